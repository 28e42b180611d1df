"""A KVCache whose tensors are given other memory, or other shapes."""
import pytest
import torch

from tests.decoder_ref import DEV, I32, BF16
from tests.test_gpu_attention import FORMS, Batch
import gemv_nvfp4_int8_amd as qp

pytestmark = pytest.mark.gpu


@FORMS
def test_tensors_that_are_given_other_memory(fp8):
    """As when a program grows or offloads its cache: a call takes the memory that the
    tensors have when it is made."""
    b = Batch([(1, 200), (4, 90)], 8, 2, 64, fp8, seed=1)
    want = b.check().clone()
    old = []
    for x in b.cache.tensors():
        new = x.clone()
        old.append(x.data)
        x.data.fill_(0x7F if x.dtype == torch.uint8 else float("nan"))
        x.data = new
    assert torch.equal(b.call(), want)
    slots = torch.tensor([3, 9], dtype=I32, device=DEV)
    before = [x.clone() for x in old]
    q = torch.empty((2, 8, 64), dtype=BF16, device=DEV)
    qp.qk_norm_rope_cache(torch.ones((2, 12 * 64), dtype=BF16, device=DEV), None, None, 1e-6, slots, None, 1.0, qp.QP_ROPE_HALF,
                          slots, b.handle, q)
    torch.cuda.synchronize()
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(old, before))
    # ones: 1, or E4M3's 448 times the F32 scale 1 / 448, which is off by half a step, 2^-24 of it
    for which in ("k", "v"):
        assert torch.all((b.cache.get(which, slots) - 1.0).abs() <= 2.0 ** -24)


@FORMS
def test_tensors_that_no_longer_fit_are_refused(fp8):
    names = ("k", "v", "k_scale", "v_scale") if fp8 else ("k", "v")
    for name in names:
        for change in ("fewer", "order", "size"):
            b = Batch([(1, 200)], 8, 2, 64, fp8, seed=1)
            x = getattr(b.handle, name)
            if change == "fewer":
                x.data = x.data[:-1].clone()
            elif change == "order":
                x.data = x.data.transpose(0, 2)
            else:
                x.resize_(len(x) + 1, *x.shape[1:])
            out = torch.full_like(b.q, 3.0)
            with pytest.raises(ValueError):
                b.call(out)
            torch.cuda.synchronize()
            assert torch.all(out == 3.0)
