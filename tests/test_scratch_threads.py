"""The workspaces that calls without one of the caller's use: one per host thread, device
and stream. A call queues kernels that hand their results on through it, and two threads'
kernels may interleave on one stream. The bookkeeping of the buffers runs here without a
GPU, on host memory; the pools and decodes of two threads on one."""
import contextlib
import threading
import types

import pytest
import torch

import gqa_decode_attention_kv_gb300 as gq


def _host_torch():
    """What the bookkeeping asks of torch, on host memory."""
    cuda = types.SimpleNamespace(stream=lambda s: contextlib.nullcontext(), current_stream=lambda d=None: None,
                                 is_current_stream_capturing=lambda: False, current_device=lambda: 0)
    return types.SimpleNamespace(cuda=cuda, uint8=torch.uint8, device=torch.device,
                                 empty=lambda n, dtype, device: torch.empty(n, dtype=dtype))


def _in_threads(n, work):
    out, errors = [None] * n, []
    start = threading.Barrier(n)

    def run(i):
        try:
            start.wait()
            out[i] = work(i)
        except BaseException as e:  # noqa: BLE001
            errors.append(e)
            start.abort()
    threads = [threading.Thread(target=run, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]
    return out


@pytest.mark.parametrize("which", ["decode", "pages"])
def test_threads_on_one_stream_get_workspaces_of_their_own(monkeypatch, which):
    monkeypatch.setattr(gq, "torch", _host_torch())
    monkeypatch.setattr(gq, "_raw_stream", lambda idx: 7)
    monkeypatch.setattr(gq, "_workspace_size_of", lambda *a: 4096)
    monkeypatch.setattr(gq, "_pages_workspace_size", lambda *a: 4096)
    dev = torch.device("cuda", 0)

    def get(_):
        if which == "decode":
            return gq.workspace_for(2, 8, 2, 64, dev)
        return gq._pages_workspace(100, 4, dev, None, None)

    def twice(i):
        a, b = get(i), get(i)
        assert a is b                                    # a thread's calls share one
        return a

    got = [t for _ in range(3) for t in _in_threads(1, twice)]        # one after the other
    got += _in_threads(2, twice)
    assert len({t.data_ptr() for t in got}) == 5


@pytest.fixture(scope="module")
def lib():
    gq._build.build()
    return gq.load()


@pytest.mark.gpu
def test_two_pools_of_two_threads_on_one_stream(lib):
    """Reservations and forks of several launches each; every pool must come out as when
    its thread has the stream to itself."""
    def work(i, rounds=60):
        rows, blocks, pages = 64, 24, 3000 + 500 * i
        refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        refs[: 7 + 900 * i] = 1                          # another first free page in every pool
        table = torch.full((rows, blocks), -1, dtype=torch.int32, device="cuda")
        lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        new = (torch.arange(rows, dtype=torch.int32) * 5 % 300 + i).cuda()
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        src = torch.arange(0, 8, dtype=torch.int32).repeat_interleave(3).cuda()
        dst = torch.arange(32, 56, dtype=torch.int32, device="cuda")
        all_rows, half = torch.arange(rows, dtype=torch.int32, device="cuda"), new.clone()
        half[32:] = 0
        seen = []
        for _ in range(rounds):
            gq.kv_pages_reserve(refs, table, lens, half, err=err)
            lens += half
            pairs = gq.kv_pages_fork(refs, table, lens, src, dst, err=err)
            seen.append((refs.clone(), table.clone(), pairs.pairs[: 24].clone(), pairs.count))
            gq.kv_pages_free(refs, table, lens, all_rows, err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        return [[t.cpu() for t in s] for s in seen], refs.cpu()

    alone = [work(0), work(1)]
    both = _in_threads(2, work)
    for (a, a_refs), (b, b_refs) in zip(alone, both):
        assert torch.equal(a_refs, b_refs)
        for x, y in zip(a, b):
            n = int(x[3][0])
            assert int(y[3][0]) == n and torch.equal(x[2][:n], y[2][:n])
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.gpu
def test_decodes_of_two_threads_on_one_stream(lib):
    import gqa_inputs as gi
    from helpers import TOL, max_abs_err
    from plain import attend_case

    def case_of(i):
        lens = [300 + 700 * i, 1200 - 500 * i, 40]
        case = gi.make_case(3, 16, 4, 128, lens, "bf16", seed=90 + i, device="cuda")
        return case, gq.cache_from_case(case)

    cases = [case_of(0), case_of(1)]

    def work(i):
        case, cache = cases[i]
        outs = [gq.gqa_decode(cache, case.q, case.block_table, case.context_lens, case.scale, window=600 * (j % 2),
                              sinks=4) for j in range(60)]
        torch.cuda.synchronize()
        return [o.cpu() for o in outs]

    for (case, _), outs in zip(cases, _in_threads(2, work)):
        for window, x in zip((0, 600), outs):
            assert max_abs_err(x, attend_case(case, window, 4)) <= TOL
        for j, x in enumerate(outs):                     # the same sums in another order at most
            assert float((x - outs[j % 2]).abs().max()) <= TOL
