"""Calls of different sizes from several host threads at once, each on a
stream and a workspace of its own: none may fail for another's size, and each
gives what it gives alone."""
import threading

import numpy as np
import pytest
import torch

import lightning_indexer_top_index_b200 as L

pytestmark = pytest.mark.gpu


def _score(dtype, H, N):
    def make(g):
        f = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float32)).cuda().to(dtype)  # noqa: E731
        q, w = f(1, 4, H, 128), torch.rand(1, 4, H, device="cuda")
        kv = L.DeviceKV(L.F32 if dtype == torch.float32 else L.BF16, 128, f(N, 128))
        out = torch.zeros(1, 4, N, device="cuda")
        return lambda stream: L.index_score(q, w, kv, N, out, stream), out
    return make


def _attn(H, n):
    def make(g):
        f = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
        q, kv = f(1, H, 512), L.DeviceKV(L.F32, 512, f(256, 512))
        ids = torch.arange(n, dtype=torch.int32, device="cuda")[None]
        out, lse = torch.zeros(1, H, 512, device="cuda"), torch.zeros(1, H, device="cuda")
        ws = L.workspace(L.workspace_size(L.OP_ATTN, L.attn_args(q, kv, 256, ids, None, None, 0, 0.04, out, lse)))
        return lambda stream: L.sparse_attn_decode(q, kv, 256, ids, scale=0.04, out=out, lse=lse, ws=ws,
                                                   stream=stream), out
    return make


def _topp(N):
    def make(g):
        p = torch.from_numpy(g.random((1, N)).astype(np.float32)).cuda()
        p /= p.sum()
        bits = torch.zeros(1, 1, (N + 31) // 32, dtype=torch.int32, device="cuda")
        ws = L.workspace(1 << 20)
        return lambda stream: L.selection_eval(L.EVAL_TOPP, N=N, probs=p, topp_bits=bits, ws=ws, stream=stream), bits
    return make


def _golden(H, N):
    def make(g):
        f = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
        q, kv = f(1, 1, H, 512), L.DeviceKV(L.F32, 512, f(N, 512))
        out = torch.zeros(1, 1, N, device="cuda")
        ws = L.workspace(1 << 20)
        return lambda stream: L.selection_eval(L.EVAL_GOLDEN, H=H, N=N, qa=q, kv=kv, probs=out, ws=ws,
                                               stream=stream), out
    return make


@pytest.mark.parametrize("makers", [
    [_score(torch.bfloat16, 32, 200), _score(torch.bfloat16, 128, 200), _score(torch.bfloat16, 96, 200)],
    [_score(torch.float32, 20, 100), _score(torch.float32, 128, 100), _score(torch.float32, 64, 100)],
    [_attn(64, 32), _attn(3, 32), _attn(40, 64)],
    [_topp(50000), _topp(1000), _topp(20000)],
    [_golden(64, 128), _golden(2, 128), _golden(30, 64)]], ids=["score-tc", "score-cc", "attention", "top-p", "golden"])
def test_different_sizes_from_several_threads(cuda_device, makers):
    g = np.random.default_rng(1)
    calls = [m(g) for m in makers]
    alone = []
    for call, out in calls:
        call(torch.cuda.current_stream())
        alone.append(out.clone())
    torch.cuda.synchronize()
    errors, start = [], threading.Barrier(len(calls))

    def work(call):
        stream = torch.cuda.Stream()
        start.wait()
        for _ in range(3000):
            try:
                call(stream)
            except Exception as e:
                errors.append(str(e))
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(call,)) for call, _ in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, f"{len(errors)} calls failed: {errors[0]}"
    for (_, out), want in zip(calls, alone):
        assert torch.equal(out, want)
