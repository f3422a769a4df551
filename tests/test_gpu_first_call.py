"""The first call of a host thread: it has no context current yet, which the
calls that make tensor maps must see to themselves."""
import threading

import numpy as np
import pytest
import torch

import lightning_indexer_top_index_b200 as L

pytestmark = pytest.mark.gpu


def _f(*shape):
    g = np.random.default_rng(len(shape))
    return torch.from_numpy(g.standard_normal(shape).astype(np.float32)).cuda().bfloat16()


def _score():
    q, w, kv = _f(1, 1, 64, 128), torch.ones(1, 1, 64, device="cuda"), L.DeviceKV(L.BF16, 128, _f(300, 128))
    out = torch.zeros(1, 1, 300, device="cuda")
    return lambda stream: L.index_score(q, w, kv, 300, out, stream), out


def _paged():
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    cache = L.PagedKV(L.DeviceKV(L.BF16, 512, _f(256, 512)), table, 64)
    call = L.paged_attn_call(_f(1, 1, 64, 512), cache, torch.full((1,), 200, dtype=torch.int32, device="cuda"))
    return call, call.out[0]


@pytest.mark.parametrize("make", [_score, _paged])
def test_first_call_of_a_thread(cuda_device, make):
    call, out = make()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    call(torch.cuda.current_stream())
    torch.cuda.synchronize()
    want, errors = out.clone(), []
    out.zero_()
    torch.cuda.synchronize()

    def work(raw):
        try:
            call(raw)
        except Exception as e:
            errors.append(str(e))

    for raw in (stream.cuda_stream, stream.cuda_stream):  # a thread each
        t = threading.Thread(target=work, args=(raw,))
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert torch.equal(out, want) and want.abs().max() > 0
