"""Argument checks of the paged calls' Python binding (no GPU): what the C ABI
cannot see, because it gets pointers."""

import pytest
import torch

from kv_cache_vector_13_b200 import api


def quantizer(d=128, **kw):
    return api.Quantizer(d, 4, "mse", device="cpu", **kw)


def cache(qz, pages=3, H=2, P=16):
    return api.empty_cache(qz, pages, H, P, device="cpu")


def calls(kq, vq, kc, vc, bad_k):
    """The calls that take this K or this V cache; none may get as far as a launch."""
    k = torch.zeros((4, 2, kq.d))
    slots = torch.zeros(4, dtype=torch.int64)
    op = object.__new__(api.PagedAttention)  # without a workspace, which needs a GPU
    op.kq, op.vq, op.Hq, op.Hkv, op.max_requests, op.max_tokens, op.device = kq, vq, 2, 2, 4, 4, -1
    op._ws, op.ws_bytes = 0, 0
    yield lambda: api.paged_append(kq, vq, k, k, kc, vc, slots)
    yield lambda: api.paged_dequant(*((kq, kc) if bad_k else (vq, vc)), slots)
    yield lambda: op(k.bfloat16(), kc, vc, torch.zeros((4, 2), dtype=torch.int32), torch.ones(4, dtype=torch.int32))


def other(c, **kw):
    return api.PackedCache(**{**dict(codes=c.codes, norms=c.norms), **kw})


@pytest.mark.parametrize("bad", [
    lambda c: other(c, codes=None),
    lambda c: other(c, codes=c.codes.float()),
    lambda c: other(c, norms=c.norms.double()),
    lambda c: other(c, codes=c.codes[:2]),                          # fewer pages
    lambda c: other(c, codes=c.codes[:, :1]),                       # fewer heads
    lambda c: other(c, codes=c.codes[:, :, :15]),                   # shorter pages
    lambda c: other(c, codes=c.codes[..., 0]),                      # no record dimension
    lambda c: other(c, codes=c.codes[..., :32]),                    # part of each record
    lambda c: other(c, codes=c.codes.transpose(2, 3).contiguous().transpose(2, 3)),
    lambda c: cache(quantizer(64)),                                 # records of another head size
    lambda c: cache(api.Quantizer(128, 3, device="cpu")),           # of another width
])
def test_caches_that_are_not_the_quantizers_are_refused(bad):
    kq, vq = quantizer(), quantizer(seed_rot=1)
    kc, vc = cache(kq), cache(vq)
    for bad_k, kx, vx in ((True, bad(kc), vc), (False, kc, bad(vc))):
        for call in calls(kq, vq, kx, vx, bad_k):
            with pytest.raises(AssertionError, match="fp32 norms and uint8 codes|are not those of|share one record layout"):
                call()


def test_tensors_of_the_host_are_refused():
    """Host addresses may not reach a launch, whatever GPU is there."""
    kq, vq = quantizer(), quantizer(seed_rot=1)
    for bad_k in (True, False):
        for call in calls(kq, vq, cache(kq), cache(vq), bad_k):
            with pytest.raises(AssertionError, match="CUDA device"):
                call()
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(AssertionError, match="CUDA device"):
        api.PagePlanner(2, 16, 8, device="cpu")(i32, i32, i32, i32[:1], torch.zeros((2, 4), dtype=torch.int32))
