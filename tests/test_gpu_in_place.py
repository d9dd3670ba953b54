"""What a call writes where it was (``out``, gradients clipped in place) counts as changed
for torch.autograd: a backward that needs the old values raises."""
import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def swz():
    return require_gpu()


def calls(swz):
    """Each call with a result of its caller's, and that result's shape and type."""
    bf16, f32 = torch.bfloat16, torch.float32
    x = torch.randn((64, 128), device="cuda").bfloat16()
    w = torch.randn((128, 128), device="cuda").bfloat16()
    q8, s8 = swz.quantize_fp8(x)
    w8, sw8 = swz.quantize_fp8(w, "square")
    qi, si = swz.quantize_int8(x)
    wi, swi = swz.quantize_int8(w)
    words = torch.randn((64, 128), device="cuda")
    return {
        "gemm": (lambda o: swz.gemm(x, w, out=o), (64, 128), f32),
        "gemm_mma_sync": (lambda o: swz.gemm_mma_sync(w, w, out=o), (128, 128), f32),
        "transpose": (lambda o: swz.transpose(words, out=o), (128, 64), f32),
        "gemm_fp8": (lambda o: swz.gemm_fp8(q8, s8, w8, sw8, out=o), (64, 128), bf16),
        "linear_fp8": (lambda o: swz.linear_fp8(x, w8, sw8, out=o), (64, 128), bf16),
        "newton_schulz": (lambda o: swz.newton_schulz(w, out=o), (128, 128), bf16),
        "newton_schulz over G": (lambda o: swz.newton_schulz(o, out=o), (128, 128), f32),
        "gemm_int8": (lambda o: swz.gemm_int8(qi, si, wi, swi, out=o), (64, 128), bf16),
        "linear_int8": (lambda o: swz.linear_int8(x, wi, swi, out=o), (64, 128), bf16),
        "linear_int8 over x": (lambda o: swz.linear_int8(o, wi, swi, out=o), (64, 128), bf16),
        "layer_norm_forward": (lambda o: swz.layer_norm_forward(x, out=o), (64, 128), bf16),
        "layer_norm_forward over x": (lambda o: swz.layer_norm_forward(o, out=o), (64, 128), f32),
        "clip_grad_norm": (lambda o: swz.clip_grad_norm([words, o], 1.0), (7, 9), f32),
        "clip_grad_norm elsewhere": (lambda o: swz.clip_grad_norm([words, words[:1]], 1.0,
                                                                  out=[torch.empty_like(words), o]), (1, 128), bf16),
    }


NAMES = ["gemm", "gemm_mma_sync", "transpose", "gemm_fp8", "linear_fp8", "newton_schulz", "newton_schulz over G",
         "gemm_int8", "linear_int8", "linear_int8 over x", "layer_norm_forward", "layer_norm_forward over x",
         "clip_grad_norm", "clip_grad_norm elsewhere"]


@pytest.mark.parametrize("name", NAMES)
def test_saved_values(swz, name):
    call, shape, dtype = calls(swz)[name]
    a = torch.randn(shape, device="cuda", requires_grad=True)
    h = (a * 0.5).to(dtype)
    loss = (h.float() if dtype == torch.float32 else h).square().sum()  # saves h
    with torch.no_grad():
        call(h.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.parametrize("name", NAMES)
def test_only_what_is_written(swz, name):
    """Operands that a call only reads do not count as changed, and inference tensors,
    which have no counter, may be written."""
    call, shape, dtype = calls(swz)[name]
    before = []
    for cell in call.__closure__:
        if isinstance(cell.cell_contents, torch.Tensor):
            before.append((cell.cell_contents, cell.cell_contents._version))
    call(torch.randn(shape, device="cuda").to(dtype))
    for t, v in before:
        # (clip_grad_norm takes `words` in place as well)
        assert (t._version > v) == (name == "clip_grad_norm")
    with torch.inference_mode():
        call(torch.randn(shape, device="cuda").to(dtype))


def test_the_host_pipeline(swz):
    a, b, c = (torch.randn((256, 256), dtype=torch.float16).pin_memory() for _ in range(3))
    c = c.float().pin_memory()
    da, db, dc = a.cuda(), b.cuda(), c.cuda()
    versions = [t._version for t in (a, b, c, da, db, dc)]
    swz.gemm_host(a, b, c, da, db, dc)
    torch.cuda.synchronize()
    assert [t._version > v for t, v in zip((a, b, c, da, db, dc), versions)] == [False, False] + [True] * 4
