"""The compiled module in front of the layer operators' binding (`-m gpu`): it makes the calls that
it should, with the binding's own results, and leaves every call with a wrong operand to the
binding, nothing written."""
import threading

import pytest
import torch

import moe_grouped_gemm_block_amd as fp8bs

pytestmark = pytest.mark.gpu
BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
layer = fp8bs.layer


def ld(n):
    return (n + 3) // 4 * 4


def operands():
    """{name: (operands by position, positions of outputs, positions that may be None)}"""
    gen = torch.Generator("cuda").manual_seed(60)
    rand = lambda *s, t=BF16: torch.randn(*s, generator=gen, device="cuda").to(t)  # noqa: E731
    codes = lambda *s: torch.zeros(s, dtype=U8, device="cuda")  # noqa: E731
    zeros = lambda *s, t=F32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    rows, k, topk, g, m, f = 50, 256, 2, 4, 40, 128
    x, res, w = rand(rows, k), rand(rows, k), rand(k, t=F32)
    xq, sx = fp8bs.quantize_1x128(x)
    ids = torch.randint(-1, g, (rows, topk), generator=gen, device="cuda")
    pos = torch.stack([torch.randperm(g * m, generator=gen, device="cuda")[:rows] for _ in range(2)], 1).to(I32)
    pos[:, 1] = -1
    rw, d, dy = torch.rand(rows, topk, generator=gen, device="cuda"), rand(g, m, k), rand(rows, k)
    gate_up, counts = rand(g, m, 2 * f), torch.tensor([0, 40, 7, 33], dtype=I32, device="cuda")
    flat, dh = rand(rows, 2 * f), rand(rows, f)
    kq, sk = fp8bs.quantize_1x128(flat)
    many = 400                                                        # (fewer need no workspace)
    ws = zeros(fp8bs.rms_norm_backward_workspace_size(many, k), t=U8)
    return {
        "rms_norm": ([x, w, res, zeros(rows, k, t=BF16), zeros(rows, k, t=BF16), codes(rows, k), zeros(k // 128, ld(rows)),
                      zeros(rows), 1e-6, None], (3, 4, 5, 6, 7), (2, 3, 4, 7)),
        "rms_norm_backward": ([rand(many, k), torch.rand(many, generator=gen, device="cuda"), w, rand(many, k),
                               zeros(many, k, t=BF16), rand(many, k), zeros(k), False, ws, None], (4, 6), (5, 6, 8)),
        "moe_dispatch": ([ids, xq, codes(g, m, k), zeros(g, t=I32), zeros(rows, topk, t=I32), zeros(g, t=I32), sx,
                          zeros(g, k // 128, ld(m)), None, None], (2, 3, 4, 5, 7), (8,)),
        "moe_combine": ([d, pos, zeros(rows, k), rw, None], (2,), (3,)),
        "moe_combine_backward": ([dy, pos, d, rw, zeros(g, m, k, t=BF16), codes(g, m, k), zeros(g, k // 128, ld(m)),
                                  zeros(rows, topk), None], (4, 5, 6, 7), (3, 4, 7)),
        "gated_quantize": ([gate_up, codes(g, m, f), zeros(g, f // 128, ld(m)), codes(g, m, 2 * f),
                            zeros(g, 2 * f // 128, ld(m)), None, counts, 0, None], (1, 2, 3, 4), (5,)),
        "gated_quantize_backward": ([kq, dh, sk, zeros(rows, 2 * f, t=BF16), codes(rows, 2 * f), zeros(2 * f // 128, ld(rows)),
                                     codes(128, 2 * f), zeros(1, 2 * f), codes(128, f), zeros(1, f), None, 1, None],
                                    tuple(range(3, 10)), (3, 10)),
        "quantize_128x1": ([xq, codes(128, k), zeros(1, k), sx, None, None], (1, 2), (4,)),
    }


def by_the_binding(name, a):
    """the same call through the binding's own checks"""
    v = list(a)
    if name.startswith("gated"):
        v[-2] = ["silu", "gelu_tanh"][v[-2]]
    order = {"rms_norm": lambda: fp8bs.fp8bs_rms_norm(*v), "rms_norm_backward": lambda: fp8bs.fp8bs_rms_norm_backward(*v),
             "moe_dispatch": lambda: fp8bs.fp8bs_moe_dispatch(*v), "moe_combine": lambda: fp8bs.fp8bs_moe_combine(*v),
             "moe_combine_backward": lambda: fp8bs.fp8bs_moe_combine_backward(*v),
             "gated_quantize": lambda: fp8bs.fp8bs_gated_quantize(*v),
             "gated_quantize_backward": lambda: fp8bs.fp8bs_gated_quantize_backward(*v),
             "quantize_128x1": lambda: fp8bs.fp8bs_quantize_128x1(*v)}
    order[name]()


NAMES = ["rms_norm", "rms_norm_backward", "moe_dispatch", "moe_combine", "moe_combine_backward", "gated_quantize",
         "gated_quantize_backward", "quantize_128x1"]


@pytest.mark.parametrize("name", NAMES)
def test_the_binding_and_the_module_agree(name, monkeypatch):
    layer._load()
    results = []
    for way in ("module", "public", "binding", "stream"):
        a, outputs, _ = operands()[name]
        if way == "module":
            assert getattr(layer._quick, name)(*a) == 0
        elif way == "public":
            by_the_binding(name, a)
        elif way == "stream":
            torch.cuda.synchronize()
            a[-1] = torch.cuda.Stream()
            by_the_binding(name, a)
            a[-1].synchronize()
        else:
            with monkeypatch.context() as m:
                m.setattr(layer, "_quick", None)
                by_the_binding(name, a)
        torch.cuda.synchronize()
        results.append([a[i].cpu() for i in outputs])
    assert any(bool((t != 0).any()) for t in results[0])
    for other in results[1:]:
        for u, v in zip(results[0], other):
            assert torch.equal(u, v)


# scales are taken in any shape that holds as many
SCALES = {"rms_norm": (6,), "moe_dispatch": (6, 7), "moe_combine_backward": (6,), "gated_quantize": (2, 4),
          "gated_quantize_backward": (2, 5, 7, 9), "quantize_128x1": (2, 3)}


@pytest.mark.parametrize("name", NAMES)
def test_wrong_operands_are_left_to_the_binding(name):
    layer._load()
    call = getattr(layer._quick, name)
    a, _, optional = operands()[name]
    for i, t in enumerate(a):
        if not isinstance(t, torch.Tensor):
            continue
        strided = torch.stack([t, t], -1)[..., 0]
        wrong = [t.cpu(), 3, "x", t.to(torch.float64), strided]
        if (name, i) == ("rms_norm_backward", 8):                     # a workspace
            assert call(*a[:i], t[:-1], *a[i + 1:]) == 3              # too small: the library's status
            wrong.append(t.view(1, -1))
        else:
            wrong += [t.reshape(-1)[:-1], torch.empty(0, dtype=t.dtype, device="cuda")]
            if i not in SCALES.get(name, ()):
                wrong.append(t[None, None])
        if i not in optional:
            wrong.append(None)
        for w in wrong:
            assert call(*a[:i], w, *a[i + 1:]) == -1, (i, w if not isinstance(w, torch.Tensor) else (w.shape, w.dtype))
    assert call(*a[:-1]) == -1 and call(*a, None) == -1 and call() == -1
    assert call(*a[:-1], "stream") == -1
    torch.cuda.synchronize()


def test_numbers_of_the_wrong_kind_are_left_to_the_binding():
    layer._load()
    a = operands()["rms_norm"][0]
    for eps in ("x", None, 1j):
        assert layer._quick.rms_norm(*a[:8], eps, None) == -1
    assert layer._quick.rms_norm(*a[:8], 0.0, None) == 1              # the library refuses it
    with pytest.raises(fp8bs.FP8BSError):
        fp8bs.fp8bs_rms_norm(*a[:8], eps=-1.0)
    a = operands()["gated_quantize"][0]
    for act in (-1, 1 << 40, "silu", None):
        assert layer._quick.gated_quantize(*a[:7], act, None) == -1
    with pytest.raises(ValueError):
        fp8bs.fp8bs_gated_quantize(*a[:7], activation="relu")


def test_parameters_views_and_a_missing_workspace():
    a = operands()
    x = a["rms_norm"][0]
    w = torch.nn.Parameter(x[1])
    assert layer._quick.rms_norm(x[0], w, *x[2:]) == 0
    v = a["rms_norm_backward"][0]
    assert layer._quick.rms_norm_backward(*v) == 0
    want = [v[4].clone(), v[6].clone()]
    for stream in (None, torch.cuda.Stream()):
        v[4].zero_(), v[6].zero_()
        torch.cuda.synchronize()
        if stream is not None:                                        # the binding allocates it
            assert layer._quick.rms_norm_backward(*v[:8], None, stream.cuda_stream) == -1
        fp8bs.fp8bs_rms_norm_backward(*v[:8], None, stream)
        torch.cuda.synchronize()
        assert torch.equal(v[4], want[0]) and torch.equal(v[6], want[1])
    whole = torch.zeros(100, 256, dtype=BF16, device="cuda")
    assert layer._quick.rms_norm(x[0], x[1], x[2], whole[25:75], *x[4:]) == 0
    torch.cuda.synchronize()
    assert torch.equal(whole[25:75], x[3]) and not bool(whole[:25].any()) and not bool(whole[75:].any())


def test_threads_at_once():
    """four host threads, each with operands and a stream of its own: the module lets go of the interpreter's lock"""
    layer._load()
    want = []
    for name in NAMES:
        a, outputs, _ = operands()[name]
        by_the_binding(name, a)
        torch.cuda.synchronize()
        want.append([a[i].clone() for i in outputs])
    sets = [operands() for _ in range(4)]
    torch.cuda.synchronize()
    errors = []

    def work(own):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    for name in NAMES:
                        by_the_binding(name, own[name][0])
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(own,)) for own in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for own in sets:
        for name, outs in zip(NAMES, want):
            a, outputs, _ = own[name]
            for i, t in zip(outputs, outs):
                assert torch.equal(a[i], t), (name, i)
