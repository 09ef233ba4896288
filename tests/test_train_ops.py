"""The training operators' C ABI without a GPU: struct layout and refusals.

Arguments are checked before any device work, so errors come out the same with
or without a GPU; the addresses below are never dereferenced."""
import ctypes
import os
import re
import subprocess

import pytest

from mixed_precision_optimizer_bf16_gb300 import bf16opt as C
from mixed_precision_optimizer_bf16_gb300 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = [0x7f0000000000 + (i << 32) for i in range(20)]      # buffers 4 GB apart


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return C.load()


def test_packed_descriptors_have_the_structs_layout():
    pytest.importorskip("torch")
    from mixed_precision_optimizer_bf16_gb300 import train_ops as ops
    for name, packed in (("distill", ops._DISTILL_T), ("norm_gate", ops._NORM_GATE_T), ("balance", ops._BALANCE_T)):
        cls = getattr(C, f"bf16opt_{name}_t")
        assert packed.size == ctypes.sizeof(cls)
        values = [i + 0.5 if t is ctypes.c_float else i + 1 for i, (_, t) in enumerate(cls._fields_)]
        d = cls(*values)
        assert cls.from_buffer_copy(packed.pack(*values)).__class__ is cls
        for f, v in zip(cls._fields_, values):
            assert getattr(cls.from_buffer_copy(packed.pack(*values)), f[0]) == getattr(d, f[0]) == v, (name, f)


def has_gpu():
    torch = pytest.importorskip("torch")
    return torch.cuda.is_available()


@pytest.mark.parametrize("name", ["distill", "norm_gate", "balance"])
def test_struct_layout_matches_header(name, tmp_path):
    cls = getattr(C, f"bf16opt_{name}_t")
    fields = [f for f, _ in cls._fields_]
    src = tmp_path / "probe.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "bf16opt.h"\nint main(void) {\nprintf("%zu", sizeof(bf16opt_' + name +
                   "_t));\n" + "".join(f'printf(" %zu", offsetof(bf16opt_{name}_t, {f}));\n' for f in fields) + "return 0; }\n")
    exe = tmp_path / "probe"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in fields]


def test_limits_match_header():
    text = open(os.path.join(ROOT, "include", "bf16opt.h")).read()
    for n in ("DISTILL_MAX_K", "NORM_MAX_HIDDEN", "BALANCE_MAX_EXPERTS", "BALANCE_MAX_K", "TYPE_F32", "INDEX_I64", "NORM_LAYER",
              "NORM_RMS", "GATE_SIGMOID"):
        assert int(re.search(rf"#define BF16OPT_{n} (\d+)", text).group(1)) == getattr(C, "BF16OPT_" + n)


def distill(**more):
    d = C.bf16opt_distill_t(8, 1000, 4, C.BF16OPT_TYPE_BF16, C.BF16OPT_TYPE_F32, 0, 1, A[0], 1000, A[1], 4, A[2], 4, A[3], A[4], A[5],
                            2.0, 1.0, 0.5)
    for n, v in more.items():
        setattr(d, n, v)
    return d


def status(rc, want, word=""):
    assert rc == want, (rc, C.bf16opt_last_error())
    if want < 0:
        assert word in C.bf16opt_last_error()


INVALID, ALIGN = C.BF16OPT_ERR_INVALID_ARG, C.BF16OPT_ERR_ALIGNMENT
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("more,word", [
    (dict(logits_type=2), "element type"), (dict(teacher_type=-1), "element type"), (dict(ids_type=5), "index type"),
    (dict(labels_type=2), "index type"), (dict(vocab=0), "vocab"), (dict(vocab=(1 << 30) + 1), "vocab"), (dict(k=1025), "k exceeds"),
    (dict(temperature=0.0), "temperature"), (dict(temperature=-1.0), "temperature"), (dict(temperature=NAN), "temperature"),
    (dict(temperature=INF), "temperature"), (dict(temperature=1e-42), "temperature"), (dict(kl_weight=-1.0), "kl_weight"),
    (dict(ce_weight=NAN), "ce_weight"), (dict(logits_stride=999), "stride"), (dict(ids_stride=3), "stride"),
    (dict(teacher_stride=0), "stride"), (dict(rows=1 << 41), "overflow"), (dict(logits_stride=1 << 62), "overflow"),
    (dict(logits=None), "NULL"), (dict(teacher_ids=None), "NULL"), (dict(teacher_logits=None), "NULL")])
def test_distill_refuses(more, word):
    d = distill(**more)
    status(C.bf16opt_distill_forward(d, A[6], A[7]), INVALID, word)
    status(C.bf16opt_distill_backward(d, A[7], A[8], A[9], 1000), INVALID, word)
    status(C.bf16opt_distill_loss_grad(d, A[8], A[6], A[7], A[9], 1000), INVALID, word)


def test_distill_refuses_outputs():
    d = distill()
    status(C.load().bf16opt_distill_forward(None, A[6], A[7], None), INVALID, "descriptor")
    status(C.bf16opt_distill_forward(d, None, A[7]), INVALID, "NULL")
    status(C.bf16opt_distill_backward(d, None, A[8], A[9], 1000), INVALID, "NULL")
    status(C.bf16opt_distill_backward(d, A[7], A[8], None, 1000), INVALID, "NULL")
    status(C.bf16opt_distill_backward(d, A[7], A[8], A[9], 999), INVALID, "stride")
    status(C.bf16opt_distill_backward(d, A[7], A[8], A[0] + 64, 1000), INVALID, "overlaps")
    status(C.bf16opt_distill_backward(d, A[7], A[8], A[0], 1008), INVALID, "overlaps")      # in place needs the same stride
    status(C.bf16opt_distill_forward(d, A[5], A[7]), INVALID, "overlaps")
    status(C.bf16opt_distill_forward(d, A[6], A[6] + 4), INVALID, "two outputs")
    status(C.bf16opt_distill_forward(d, A[6] + 2, A[7]), ALIGN)
    status(C.bf16opt_distill_backward(d, A[7], A[8], A[9] + 1, 1000), ALIGN)
    for field, off in (("logits", 1), ("teacher_ids", 2), ("teacher_logits", 2), ("teacher_lse", 1), ("labels", 4), ("row_weight", 2)):
        status(C.bf16opt_distill_forward(distill(**{field: getattr(d, field) + off}), A[6], A[7]), ALIGN)
    status(C.bf16opt_distill_forward(distill(rows=0, logits=None), None, None), C.BF16OPT_OK)


def norm(**more):
    d = C.bf16opt_norm_gate_t(12, 64, C.BF16OPT_TYPE_BF16, C.BF16OPT_TYPE_BF16, C.BF16OPT_TYPE_BF16, C.BF16OPT_NORM_LAYER,
                              C.BF16OPT_NORM_RMS, 0, 0, 4, A[0], A[1], A[2], A[3], None, 1.0, 1.0, 1e-5)
    for n, v in more.items():
        setattr(d, n, v)
    return d


def norm_forward(d, x=A[5], y=A[6], r=A[7], h=A[8], stats=A[9]):
    return C.bf16opt_norm_gate_forward(d, x, y, r, h, stats)


def norm_backward(d, **more):
    a = dict(dr=A[5], dh=A[6], r=A[7], y=A[8], stats=A[9], dx=A[10], dy=A[11], dgate=A[12], dpre_weight=A[13], dpre_bias=A[14],
             dpost_weight=A[15], dpost_bias=None, workspace=A[16], workspace_bytes=1 << 31)
    a.update(more)
    return C.bf16opt_norm_gate_backward(d, **a)


@pytest.mark.parametrize("more,word", [
    (dict(branch_type=3), "element type"), (dict(stream_type=-2), "element type"), (dict(weight_type=9), "element type"),
    (dict(branch_type=C.BF16OPT_TYPE_F32), "FP32 stream"), (dict(hidden=0), "hidden"), (dict(hidden=16385), "hidden"),
    (dict(pre=3), "norm"), (dict(post=-1), "norm"), (dict(gate_act=2), "gate_act"), (dict(reserved=1), "reserved"),
    (dict(gate=None), "gate_rows"), (dict(gate_rows=0), "gate_rows"), (dict(gate_rows=5), "divide"), (dict(gate_rows=24), "divide"),
    (dict(pre=0), "weight without"), (dict(post=0), "weight without"), (dict(eps=0.0), "eps"), (dict(eps=NAN), "eps"),
    (dict(residual_scale=INF), "finite"), (dict(branch_scale=NAN), "finite"), (dict(rows=1 << 40), "rows")])
def test_norm_refuses(more, word):
    d = norm(**more)
    status(norm_forward(d), INVALID, word)
    status(C.bf16opt_norm_gate_workspace(d)[0], INVALID, word)
    status(norm_backward(d), INVALID, word)


def test_norm_refuses_pointers():
    d = norm()
    for n in ("x", "y", "r", "h"):
        status(norm_forward(d, **{n: None}), INVALID, "NULL")
    status(norm_forward(d, r=A[5] + 32), INVALID, "overlaps")
    status(norm_forward(d, r=A[6]), INVALID, "overlaps")
    status(norm_forward(d, h=A[7]), INVALID, "outputs overlap")
    status(norm_forward(d, x=A[5] + 1), ALIGN)
    status(norm_forward(norm(gate=A[0] + 1)), ALIGN)
    status(norm_forward(norm(pre_bias=A[2] + 1)), ALIGN)
    status(norm_forward(norm(pre=0, pre_weight=None, pre_bias=None)), INVALID, "h without")
    for n in ("y", "dx", "dy", "stats"):
        status(norm_backward(d, **{n: None}), INVALID, "NULL")
    status(norm_backward(d, r=None), INVALID, "NULL")
    status(norm_backward(d, dpost_bias=A[17]), INVALID, "not there")
    status(norm_backward(d, dx=A[10] + 1), ALIGN)
    status(norm_backward(d, workspace=A[16] + 8), ALIGN)


def balance(**more):
    d = C.bf16opt_balance_t(256, 16, 2, 4, C.BF16OPT_TYPE_F32, 1, A[0], 16, A[1], 0.01, 0.001)
    for n, v in more.items():
        setattr(d, n, v)
    return d


@pytest.mark.parametrize("more,word", [
    (dict(logits_type=4), "element type"), (dict(experts=0), "experts"), (dict(experts=1025, logits_stride=1025), "experts"),
    (dict(k=0), "k must"), (dict(k=17), "k must"), (dict(experts=64, logits_stride=64, k=33), "k must"), (dict(groups=0), "divide"),
    (dict(groups=3), "divide"), (dict(groups=512), "divide"), (dict(logits_stride=15), "stride"), (dict(renormalise=2), "renormalise"),
    (dict(balance_weight=-0.1), "balance_weight"), (dict(z_weight=NAN), "z_weight"), (dict(tokens=1 << 40), "tokens"),
    (dict(tokens=1 << 33, groups=1), "2^31")])
def test_balance_refuses(more, word):
    d = balance(**more)
    status(C.bf16opt_balance_workspace(d)[0], INVALID, word)
    status(C.bf16opt_balance_forward(d, A[2], A[3], A[4], A[5], A[6], A[7], 1 << 30), INVALID, word)
    status(C.bf16opt_balance_backward(d, A[2], A[4], A[6], A[3], A[5], A[8], 16), INVALID, word)


def test_balance_refuses_pointers():
    d = balance()
    for i in range(5):
        a = A[2:7]
        a[i] = None
        status(C.bf16opt_balance_forward(d, *a, A[7], 1 << 30), INVALID, "NULL")
    status(C.bf16opt_balance_forward(balance(logits=None), *A[2:7], A[7], 1 << 30), INVALID, "NULL")
    status(C.bf16opt_balance_forward(d, A[2] + 1, *A[3:7], A[7], 1 << 30), ALIGN)
    status(C.bf16opt_balance_forward(d, *A[2:7], A[7] + 4, 1 << 30), ALIGN)
    status(C.bf16opt_balance_backward(d, A[2], A[4], A[6], A[3], A[5], A[8], 15), INVALID, "stride")
    status(C.bf16opt_balance_backward(d, A[2], A[4], A[6], A[3], A[5], A[0] + 4, 16), INVALID, "overlaps")
    status(C.bf16opt_balance_backward(d, A[2], A[4], A[6], A[3], A[5], None, 16), INVALID, "NULL")


def test_without_a_device():
    if has_gpu():
        pytest.skip("a CUDA device is present")
    status(C.bf16opt_distill_forward(distill(), A[6], A[7]), C.BF16OPT_ERR_UNSUPPORTED, "no CUDA device")
    status(norm_forward(norm()), C.BF16OPT_ERR_UNSUPPORTED, "no CUDA device")
    status(C.bf16opt_norm_gate_workspace(norm())[0], C.BF16OPT_ERR_UNSUPPORTED, "no CUDA device")
    status(C.bf16opt_balance_workspace(balance())[0], C.BF16OPT_ERR_UNSUPPORTED, "no CUDA device")


def test_python_layer_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    from mixed_precision_optimizer_bf16_gb300 import train_ops as ops
    z = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        ops.distill_forward(z, z.int(), z)
    with pytest.raises(ValueError, match="CUDA"):
        ops.norm_gate_forward(z, z)
    with pytest.raises(ValueError, match="CUDA"):
        ops.balance_forward(z, 2)


def test_reference_gradients_against_differences():
    """The 64-bit reference that the GPU tests compare with is itself checked."""
    torch = pytest.importorskip("torch")
    import train_ops_reference as R
    g = torch.Generator().manual_seed(0)
    rnd = lambda *s: torch.randn(*s, dtype=torch.float64, generator=g)  # noqa: E731
    z, ids, top = 2 * rnd(3, 20), torch.randint(-1, 21, (3, 5), generator=g), rnd(3, 5)
    ids[0, 1] = ids[0, 2] = 7
    how = dict(temperature=1.7, kl_weight=0.6, ce_weight=0.4, labels=torch.tensor([7, -100, 3]), row_weight=torch.tensor([1.0, 0.5, 2.0]))
    for extra in ({}, {"teacher_lse": torch.tensor([2.0, 2.5, 3.0])}):
        v = rnd(3, 20)
        d = (R.distill(z + 1e-6 * v, ids, top, **how, **extra)[0].sum() - R.distill(z - 1e-6 * v, ids, top, **how, **extra)[0].sum()) / 2e-6
        assert abs(float((R.distill(z, ids, top, **how, **extra)[1] * v).sum() - d)) < 1e-7
    z, up, v = rnd(30, 6), rnd(30, 2), rnd(30, 6)
    for renorm in (True, False):
        def value(s):
            _, w, _, l, _ = R.balance(z + s * v, 2, groups=3, balance_weight=0.5, z_weight=0.1, renormalise=renorm)
            return l + (w * up).sum()
        dz = R.balance(z, 2, groups=3, balance_weight=0.5, z_weight=0.1, renormalise=renorm, dweights=up)[4]
        assert abs(float((dz * v).sum() - (value(1e-7) - value(-1e-7)) / 2e-7)) < 1e-6
    x, y = rnd(6, 9), rnd(6, 9)
    par = dict(pre_weight=rnd(9), pre_bias=rnd(9), post_weight=rnd(9), post_bias=rnd(9), gate=rnd(3, 9))
    rest = dict(pre="layer", post="rms", gate_act="sigmoid", residual_scale=0.7, branch_scale=1.1)
    cr, ch = rnd(6, 9), rnd(6, 9)
    got = R.norm_gate_backward(cr, ch, R.norm_gate(x, y, **rest, **par)[0], y, **rest, **par)
    for n in ("x", "y", *par):
        v = rnd(*{"x": x, "y": y, **par}[n].shape)
        def value(s):
            m = {k: t + (s * v if k == n else 0) for k, t in {"x": x, "y": y, **par}.items()}
            r, h, _ = R.norm_gate(**m, **rest)
            return (r * cr).sum() + (h * ch).sum()
        assert abs(float((got["d" + n] * v).sum() - (value(1e-6) - value(-1e-6)) / 2e-6)) < 1e-6, n
