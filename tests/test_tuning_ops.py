"""The fine-tuning operators' C ABI without a GPU: struct layout and refusals, and the plain references themselves.

Arguments are checked before any device work, so errors come out the same with
or without a GPU; the addresses below are never dereferenced."""
import ctypes
import math
import os
import re
import subprocess

import pytest

from mixed_precision_optimizer_bf16_gb300 import bf16opt as C
from mixed_precision_optimizer_bf16_gb300 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = [0x7f0000000000 + (i << 33) for i in range(20)]      # buffers 8 GB apart
INVALID, ALIGN = C.BF16OPT_ERR_INVALID_ARG, C.BF16OPT_ERR_ALIGNMENT
NAN, INF = float("nan"), float("inf")
NAMES = ["tokens", "policy", "preference", "pack", "glu", "rotary"]


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return C.load()


@pytest.mark.parametrize("name", NAMES)
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


@pytest.mark.parametrize("name", NAMES)
def test_packed_descriptors_have_the_structs_layout(name):
    pytest.importorskip("torch")
    from mixed_precision_optimizer_bf16_gb300 import train_ops as ops
    cls, packed = getattr(C, f"bf16opt_{name}_t"), getattr(ops, f"_{name.upper()}_T")
    assert packed.size == ctypes.sizeof(cls)
    flat, n = [], 0
    for f, t in cls._fields_:
        for _ in range(getattr(t, "_length_", 1)):
            n += 1
            flat.append(n + 0.5 if t is ctypes.c_float else n)
    got, at = cls.from_buffer_copy(packed.pack(*flat)), 0
    for f, t in cls._fields_:
        v, k = getattr(got, f), getattr(t, "_length_", 1)
        assert (list(v) if k > 1 else [v]) == flat[at:at + k], f
        at += k


def test_limits_match_header():
    text = open(os.path.join(ROOT, "include", "bf16opt.h")).read()
    for n in ("TOKENS_MAX_ROWS", "PREFER_SIGMOID", "PREFER_HINGE", "PREFER_IPO", "PREFER_MAX_PAIRS", "PACK_RUN", "GLU_SILU", "GLU_GELU",
              "ROTARY_HALF", "ROTARY_INTERLEAVED", "ROTARY_MAX_DIM"):
        assert int(re.search(rf"#define BF16OPT_{n} (\w+)", text).group(1), 0) == getattr(C, "BF16OPT_" + n)


def status(rc, want, word=""):
    assert rc == want, (rc, C.bf16opt_last_error())
    if want < 0:
        assert word in C.bf16opt_last_error()


def has_gpu():
    return pytest.importorskip("torch").cuda.is_available()


# ------------------------------------------------------------------ token losses

def tokens(**more):
    d = C.bf16opt_tokens_t(8, 1000, C.BF16OPT_TYPE_BF16, 1, 1.5, A[0], 1000, A[1], A[2])
    for n, v in more.items():
        setattr(d, n, v)
    return d


BAD_TOKENS = [(dict(logits_type=2), "element type"), (dict(labels_type=-1), "index type"), (dict(vocab=0), "vocab"), (dict(vocab=(1 << 30) + 1), "vocab"),
              (dict(rows=1 << 31), "rows"), (dict(temperature=0.0), "temperature"), (dict(temperature=-1.0), "temperature"),
              (dict(temperature=NAN), "temperature"), (dict(temperature=INF), "temperature"), (dict(temperature=1e-39), "temperature"),
              (dict(logits_stride=999), "stride"), (dict(rows=(1 << 31) - 1, logits_stride=1 << 40), "sizes"), (dict(logits=None), "NULL"),
              (dict(labels=None), "NULL")]


@pytest.mark.parametrize("more,word", BAD_TOKENS)
def test_tokens_refusals(more, word):
    d = tokens(**more)
    status(C.bf16opt_token_logp_forward(d, A[3], A[4]), INVALID, word)
    status(C.bf16opt_token_logp_backward(d, A[4], A[5], 8, A[6], 1000), INVALID, word)
    p = C.bf16opt_policy_t(A[7], A[8], A[9], 0.2, 0.2, 0.1, 0)
    status(C.bf16opt_policy_forward(d, p, A[3], A[4], A[5]), INVALID, word)
    status(C.bf16opt_policy_loss_grad(d, p, None, A[3], A[4], A[6], 1000), INVALID, word)
    q = C.bf16opt_preference_t(2, 0, 0, A[10], A[11], 0.1, 0.0, 0.0, 0)
    d.row_weight = None
    status(C.bf16opt_preference_forward(d, q, A[3], A[4], A[5]), INVALID, word)


@pytest.mark.parametrize("more", [dict(logits=A[0] + 1), dict(labels=A[1] + 4), dict(row_weight=A[2] + 2)])
def test_tokens_alignment(more):
    status(C.bf16opt_token_logp_forward(tokens(**more), A[3], A[4]), ALIGN, "aligned")


def test_token_logp_outputs():
    d = tokens()
    status(C.bf16opt_token_logp_forward(None, A[3], A[4]), INVALID, "descriptor")
    status(C.bf16opt_token_logp_forward(d, None, A[4]), INVALID, "NULL")
    status(C.bf16opt_token_logp_forward(d, A[3] + 1, A[4]), ALIGN, "aligned")
    status(C.bf16opt_token_logp_forward(d, A[3], A[4] + 4), ALIGN, "16-byte")
    for p in (A[0] + 8 * 2000 - 4, A[1], A[2] + 28):
        status(C.bf16opt_token_logp_forward(d, p, A[4]), INVALID, "overlaps an input")
    status(C.bf16opt_token_logp_forward(d, A[4] + 64, A[4]), INVALID, "two outputs")
    status(C.bf16opt_token_logp_forward(tokens(rows=0, logits=None, labels=None), None, None), 0)


def test_token_logp_backward_outputs():
    d = tokens()
    status(C.bf16opt_token_logp_backward(d, None, A[5], 8, A[6], 1000), INVALID, "saved")
    status(C.bf16opt_token_logp_backward(d, A[4] + 4, A[5], 8, A[6], 1000), ALIGN, "16-byte")
    status(C.bf16opt_token_logp_backward(d, A[4], A[5], 8, None, 1000), INVALID, "dlogits")
    status(C.bf16opt_token_logp_backward(d, A[4], A[5], 8, A[6], 999), INVALID, "stride")
    status(C.bf16opt_token_logp_backward(d, A[4], A[5] + 2, 8, A[6], 1000), ALIGN, "aligned")
    status(C.bf16opt_token_logp_backward(d, A[4], A[5], 1 << 31, A[6], 1000), INVALID, "losses")
    status(C.bf16opt_token_logp_backward(d, A[4], A[5], 8, A[0], 1001), INVALID, "overlaps an input")      # another stride
    status(C.bf16opt_token_logp_backward(d, A[4], A[5], 8, A[0] + 2, 1000), INVALID, "overlaps an input")
    status(C.bf16opt_token_logp_backward(d, A[4], A[5], 8, A[4] + 64, 1000), INVALID, "overlaps an input")
    status(C.bf16opt_token_logp_backward(d, A[4], A[5], 8, A[5] + 30, 1000), INVALID, "overlaps an input")


@pytest.mark.parametrize("more,word", [(dict(clip_low=-0.1), "clip"), (dict(clip_low=1.1), "clip"), (dict(clip_low=NAN), "clip"),
                                       (dict(clip_high=-0.1), "clip"), (dict(clip_high=NAN), "clip"), (dict(kl_weight=-1.0), "kl_weight"),
                                       (dict(kl_weight=INF), "kl_weight"), (dict(reserved=1), "reserved"), (dict(advantage=None), "NULL")])
def test_policy_refusals(more, word):
    d, p = tokens(), C.bf16opt_policy_t(A[7], A[8], A[9], 0.2, 0.2, 0.1, 0)
    for n, v in more.items():
        setattr(p, n, v)
    status(C.bf16opt_policy_forward(d, p, A[3], A[4], A[5]), INVALID, word)
    status(C.bf16opt_policy_loss_grad(d, p, None, A[3], A[4], A[6], 1000), INVALID, word)


def test_policy_outputs():
    d, p = tokens(), C.bf16opt_policy_t(A[7], A[8], A[9], 0.2, INF, 0.1, 0)
    status(C.bf16opt_policy_forward(d, None, A[3], A[4], A[5]), INVALID, "descriptor")
    status(C.bf16opt_policy_forward(d, p, None, A[4], A[5]), INVALID, "NULL")
    status(C.bf16opt_policy_forward(d, p, A[3], None, A[5]), INVALID, "NULL")
    status(C.bf16opt_policy_forward(d, p, A[3], A[4], A[5] + 8), ALIGN, "16-byte")
    for x in (A[7], A[8] + 31, A[9] + 4):
        status(C.bf16opt_policy_forward(d, p, x & ~3, A[4], A[5]), INVALID, "overlaps an input")
    status(C.bf16opt_policy_loss_grad(d, p, A[10], A[10], A[4], A[6], 1000), INVALID, "overlaps an input")
    status(C.bf16opt_policy_loss_grad(d, p, A[10], A[3], A[6] + 32, A[6], 1000), INVALID, "two outputs")
    status(C.bf16opt_policy_loss_grad(d, p, A[10], A[3], A[4], None, 1000), INVALID, "dlogits")


@pytest.mark.parametrize("more,word", [(dict(pairs=65537), "pairs"), (dict(offsets_type=2), "index type"), (dict(kind=3), "kind"), (dict(kind=-1), "kind"),
                                       (dict(offsets=None), "NULL"), (dict(beta=0.0), "beta"), (dict(beta=INF), "beta"), (dict(beta=1e-40), "beta"),
                                       (dict(label_smoothing=0.6), "label_smoothing"), (dict(label_smoothing=-0.1), "label_smoothing"),
                                       (dict(label_smoothing=NAN), "label_smoothing"), (dict(margin=INF), "margin"), (dict(length_normalise=2), "length_normalise")])
def test_preference_refusals(more, word):
    d, q = tokens(row_weight=None), C.bf16opt_preference_t(2, 0, 0, A[10], A[11], 0.1, 0.0, 0.0, 0)
    for n, v in more.items():
        setattr(q, n, v)
    status(C.bf16opt_preference_forward(d, q, A[3], A[4], A[5]), INVALID, word)


def test_preference_outputs():
    d, q = tokens(row_weight=None), C.bf16opt_preference_t(2, 1, 0, A[10], A[11], 0.1, 0.0, 0.0, 0)
    status(C.bf16opt_preference_forward(tokens(), q, A[3], A[4], A[5]), INVALID, "row_weight")
    status(C.bf16opt_preference_forward(d, None, A[3], A[4], A[5]), INVALID, "descriptor")
    status(C.bf16opt_preference_forward(d, q, None, A[4], A[5]), INVALID, "NULL")
    status(C.bf16opt_preference_forward(d, q, A[3], A[4], None), INVALID, "saved")
    status(C.bf16opt_preference_forward(d, q, A[3], A[4], A[5] + 4), ALIGN, "16-byte")
    q.offsets = A[10] + 4
    status(C.bf16opt_preference_forward(d, q, A[3], A[4], A[5]), ALIGN, "aligned")
    q.offsets = A[10]
    for x in (A[10] + 36, A[11] + 12, A[0]):
        status(C.bf16opt_preference_forward(d, q, x, A[4], A[5]), INVALID, "overlaps an input")
    status(C.bf16opt_preference_forward(d, q, A[3], A[3] + 4, A[5]), INVALID, "two outputs")


# ------------------------------------------------------------------ 8 bits

def test_pack_refusals():
    d = C.bf16opt_pack_t(4, 100, C.BF16OPT_TYPE_BF16)
    for call in (lambda d, x=A[0], s=100, c=A[1], k=A[2]: C.bf16opt_pack(d, x, s, c, k),
                 lambda d, x=A[0], s=100, c=A[1], k=A[2]: C.bf16opt_unpack(d, c, k, x, s)):
        status(call(None), INVALID, "descriptor")
        status(call(C.bf16opt_pack_t(4, 0, 0)), INVALID, "columns")
        status(call(C.bf16opt_pack_t(4, (1 << 30) + 1, 0)), INVALID, "columns")
        status(call(C.bf16opt_pack_t(4, 100, 5)), INVALID, "element type")
        status(call(C.bf16opt_pack_t(1 << 50, 100, 0)), INVALID, "sizes")
        status(call(d, s=99), INVALID, "stride")
        status(call(d, s=1 << 62), INVALID, "sizes")
        for n in "xck":
            status(call(d, **{n: None}), INVALID, "NULL")
        status(call(d, x=A[0] + 1), ALIGN, "aligned")
        status(call(d, c=A[1] + 8), ALIGN, "16-byte")
        status(call(d, c=A[0] + 512), INVALID, "overlap")
        status(call(d, k=A[0] + 796), INVALID, "overlap")
        status(call(C.bf16opt_pack_t(0, 100, 0), x=None, c=None, k=None), 0)
    status(C.bf16opt_pack(d, A[0], 100, A[1], A[1] + 16), INVALID, "overlap")


def glu(**more):
    d = C.bf16opt_glu_t(4, 100, C.BF16OPT_TYPE_F32, C.BF16OPT_GLU_SILU, 1)
    for n, v in more.items():
        setattr(d, n, v)
    return d


def forward(d, gate=A[0], up=A[1], h=A[2], codes=A[3], scales=A[4], gs=100, us=100, hs=100):
    return C.bf16opt_glu_forward(d, gate, gs, up, us, h, hs, codes, scales)


def backward(d, dh=A[0], codes=A[3], scales=A[4], dgate=A[5], dup=A[6], h=A[7], ds=100, gs=100, us=100, hs=100):
    return C.bf16opt_glu_backward(d, dh, ds, codes, scales, dgate, gs, dup, us, h, hs)


@pytest.mark.parametrize("call", [forward, backward])
def test_glu_refusals(call):
    status(call(None), INVALID, "descriptor")
    for more, word in ((dict(columns=0), "columns"), (dict(type=2), "element type"), (dict(act=2), "activation"), (dict(gated=2), "gated"),
                       (dict(rows=1 << 41), "sizes"), (dict(gated=0), "NULL without")):
        status(call(glu(**more)), INVALID, word)
    status(call(glu(), gs=99), INVALID, "stride")
    status(call(glu(), us=99), INVALID, "stride")
    status(call(glu(), hs=99), INVALID, "stride")
    status(call(glu(), codes=A[3] + 1), ALIGN, "16-byte")
    status(call(glu(), codes=None), INVALID)
    status(call(glu(), scales=None), INVALID)
    status(call(glu(rows=0)), 0)


def test_glu_overlaps():
    status(forward(glu(), gate=None), INVALID, "NULL")
    status(forward(glu(), up=None), INVALID, "NULL")
    status(forward(glu(), h=None), INVALID, "NULL")
    status(forward(glu(), gate=A[0] + 2), ALIGN, "aligned")
    status(forward(glu(), h=A[0] + 4), INVALID, "overlaps an input")
    status(forward(glu(), h=A[0], hs=101), INVALID, "overlaps an input")
    status(forward(glu(), h=A[3] + 64), INVALID, "kept")
    status(forward(glu(), codes=A[0] + 64), INVALID, "kept")
    status(forward(glu(), scales=A[3] + 64), INVALID, "two outputs")
    status(backward(glu(), dgate=None), INVALID, "NULL")
    status(backward(glu(), dup=None), INVALID, "NULL")
    status(backward(glu(), dh=None), INVALID, "NULL")
    status(backward(glu(), dgate=A[0] + 4), INVALID, "overlaps an input")
    status(backward(glu(), dgate=A[0], gs=104), INVALID, "overlaps an input")
    status(backward(glu(), dgate=A[5], dup=A[5] + 4), INVALID, "two outputs")
    status(backward(glu(), dgate=A[5], dup=A[5] + 396, gs=200, us=200), INVALID, "two outputs")      # halves that meet by one element
    status(backward(glu(), dgate=A[5], dup=A[5] + 400, gs=199, us=199), INVALID, "two outputs")
    status(backward(glu(), dgate=A[5], dup=A[5] + 400, gs=200, us=201), INVALID, "two outputs")
    status(backward(glu(), h=A[3]), INVALID, "kept")
    if not has_gpu():   # what is allowed comes as far as the device
        for rc in (forward(glu()), forward(glu(), codes=None, scales=None), forward(glu(), h=A[0]), forward(glu(), h=A[1]),
                   forward(glu(gated=0), up=None), forward(glu(), gate=A[0], up=A[0] + 400, gs=200, us=200),
                   backward(glu()), backward(glu(), dgate=A[0]), backward(glu(), dup=A[0]), backward(glu(), h=A[0]), backward(glu(), h=None),
                   backward(glu(), dgate=A[5], dup=A[5] + 400, gs=200, us=200), backward(glu(), dgate=A[5] + 400, dup=A[5], gs=200, us=200),
                   backward(glu(gated=0), dup=None)):
            status(rc, C.BF16OPT_ERR_UNSUPPORTED)


# ------------------------------------------------------------------ rotary positions

FREQUENCIES = (ctypes.c_double * 128)(*([0.5] * 128))


def rotary(**more):
    """Two sequences of eight tokens, four heads and two, 64 elements of which 32 turn; q and k of their own."""
    d = C.bf16opt_rotary_t(2, 8, 4, 2, 64, 32, C.BF16OPT_TYPE_BF16, 0, 1, 0, A[4], 8, 0, ctypes.addressof(FREQUENCIES), 1.0, 0)
    for n in ("q", "out_q"):
        setattr(d, n + "_stride", (ctypes.c_uint64 * 3)(8 * 256, 256, 64))
    for n in ("k", "out_k"):
        setattr(d, n + "_stride", (ctypes.c_uint64 * 3)(8 * 128, 128, 64))
    for n, v in more.items():
        setattr(d, n, (ctypes.c_uint64 * 3)(*v) if isinstance(v, tuple) else v)
    return d


def turn(d, q=A[0], k=A[1], oq=A[2], ok=A[3]):
    return C.bf16opt_rotary(d, q, k, oq, ok)


BROKEN = (ctypes.c_double * 128)(*([0.5] * 7 + [NAN] + [0.5] * 120))


@pytest.mark.parametrize("more,word", [
    (dict(type=3), "element type"), (dict(positions_type=2), "index type"), (dict(layout=2), "layout"), (dict(inverse=2), "inverse"),
    (dict(reserved=1), "reserved"), (dict(heads=0), "heads"), (dict(heads=1 << 21), "heads"), (dict(kv_heads=1 << 21), "heads"), (dict(dim=0), "dim"),
    (dict(dim=70000), "dim"), (dict(rotary_dim=0), "rotary_dim"), (dict(rotary_dim=31), "rotary_dim"), (dict(rotary_dim=66), "rotary_dim"),
    (dict(dim=512, rotary_dim=258), "rotary_dim"), (dict(scale=INF), "scale"), (dict(scale=NAN), "scale"), (dict(frequencies=None), "frequencies"),
    (dict(frequencies=ctypes.addressof(BROKEN)), "frequency"), (dict(batch=1 << 30, seq=1 << 30), "sizes"), (dict(positions_stride=7), "positions_stride"),
    (dict(q_stride=(1 << 62, 256, 64)), "sizes"), (dict(out_q_stride=(1 << 61, 1 << 61, 64)), "sizes"),
    (dict(out_q_stride=(2048, 0, 64)), "twice"), (dict(out_q_stride=(2048, 256, 63)), "twice"), (dict(out_k_stride=(0, 128, 64)), "twice"),
    (dict(out_q_stride=(2048, 255, 64)), "twice")])
def test_rotary_refusals(more, word):
    status(turn(rotary(**more)), INVALID, word)


def test_rotary_pointers():
    status(turn(None), INVALID, "descriptor")
    for n in ("q", "k", "oq", "ok"):
        status(turn(rotary(), **{n: None}), INVALID, "NULL")
        status(turn(rotary(), **{n: A[6] + 1}), ALIGN, "aligned")
    status(turn(rotary(positions=A[4] + 4)), ALIGN, "positions")
    status(turn(rotary(), oq=A[0] + 16), INVALID, "overlaps an input")
    status(turn(rotary(), oq=A[1]), INVALID, "overlaps an input")
    status(turn(rotary(), ok=A[0]), INVALID, "overlaps an input")
    status(turn(rotary(), oq=A[4] + 64), INVALID, "overlaps an input")
    status(turn(rotary(), ok=A[2] + 512), INVALID, "two outputs")
    status(turn(rotary(out_q_stride=(4096, 512, 64)), oq=A[0]), INVALID, "overlaps an input")       # in place with other strides
    status(turn(rotary(batch=0)), 0)
    status(turn(rotary(seq=0)), 0)


def test_rotary_parts_of_one_matrix():
    """q and k as parts of one projection, in place: their spans meet, their elements do not."""
    one = dict(q_stride=(8 * 512, 512, 64), k_stride=(8 * 512, 512, 64), out_q_stride=(8 * 512, 512, 64), out_k_stride=(8 * 512, 512, 64))
    heads_first = {n: (7 * 512, 64, 512) for n in one}
    far = A[0] + 2 * 256
    status(turn(rotary(**one), k=far - 2 * 64, oq=A[0], ok=far - 2 * 64), INVALID, "overlaps an input")    # one head of both
    status(turn(rotary(**one), k=A[0] + 2 * 448, oq=A[0], ok=A[0] + 2 * 448), INVALID, "overlaps an input")    # k's last head is the next token's
    status(turn(rotary(**one), oq=A[2], ok=A[2] + 2 * 192), INVALID, "two outputs")
    if not has_gpu():
        for rc in (turn(rotary()), turn(rotary(), oq=A[0], ok=A[1]), turn(rotary(**one), k=far, oq=A[0], ok=far), turn(rotary(**one), oq=A[2], ok=A[2] + 2 * 256),
                   turn(rotary(**one), oq=A[2] + 2 * 256, ok=A[2]), turn(rotary(batch=1, **one), k=far, oq=A[0], ok=far),
                   turn(rotary(seq=1, positions_stride=0, **one), k=far, oq=A[0], ok=far), turn(rotary(kv_heads=0), k=None, ok=None),
                   turn(rotary(seq=1, positions_stride=0, batch=1, **one), k=far, oq=A[0], ok=far),
                   turn(rotary(**heads_first), k=A[0] + 2 * 4 * 512, oq=A[0], ok=A[0] + 2 * 4 * 512), turn(rotary(q_stride=(0, 256, 0))), 
                   turn(rotary(positions=None, positions_stride=0)), turn(rotary(positions_stride=0))):
            status(rc, C.BF16OPT_ERR_UNSUPPORTED)


# ------------------------------------------------------------------ the references themselves

def test_reference_gradients_against_differences():
    torch = pytest.importorskip("torch")
    import tuning_reference as R
    g = torch.Generator().manual_seed(0)
    z = torch.randn(6, 9, generator=g, dtype=torch.float64)
    labels = torch.tensor([3, 0, 8, -100, 5, 2])
    old, ref = -2 + 0.2 * torch.randn(6, generator=g), -2 + 0.2 * torch.randn(6, generator=g)
    adv, w, up = torch.randn(6, generator=g), torch.tensor([1.0, 0.5, 2.0, 1.0, 0.0, 1.0]), 0.3 + torch.rand(6, generator=g)
    offsets = torch.tensor([0, 2, 3, 3, 6])
    how = dict(temperature=1.3)

    def each(z):
        yield (R.token_logp(z, labels, row_weight=w, dloss=up, **how)[0] * up).sum(), R.token_logp(z, labels, row_weight=w, dloss=up, **how)[1]
        p = dict(old_logp=old, ref_logp=ref, clip_low=0.1, clip_high=0.3, kl_weight=0.2, row_weight=w, dloss=up, **how)
        yield (R.policy(z, labels, adv, **p)[0] * up).sum(), R.policy(z, labels, adv, **p)[3]
        for kind in ("sigmoid", "hinge", "ipo"):
            for mean in (False, True):
                q = dict(kind=kind, beta=0.7, label_smoothing=0.2, margin=0.1, length_normalise=mean, dloss=up[:2], **how)
                yield (R.preference(z, labels, offsets, **q)[0] * up[:2]).sum(), R.preference(z, labels, offsets, **q)[2]

    grads = [d for _, d in each(z)]
    for r in range(6):
        for j in (0, 3, 8):
            e = torch.zeros_like(z)
            e[r, j] = 1e-6
            for d, (above, _), (below, _) in zip(grads, each(z + e), each(z - e)):
                assert abs(float(above - below) / 2e-6 - float(d[r, j])) < 1e-7


def test_reference_activations_against_differences():
    torch = pytest.importorskip("torch")
    import tuning_reference as R
    g = torch.linspace(-9, 9, 1001, dtype=torch.float64)
    for kind in ("silu", "gelu"):
        a, slope, _ = R.act(g, kind)
        assert ((R.act(g + 1e-6, kind)[0] - R.act(g - 1e-6, kind)[0]) / 2e-6 - slope).abs().max() < 1e-8
        plain = torch.nn.functional.silu(g) if kind == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
        assert (a - plain).abs().max() < 1e-14


def test_reference_codes():
    torch = pytest.importorskip("torch")
    import tuning_reference as R
    numbers = R.e4m3_numbers()
    assert numbers[126] == 448 and numbers[1] == 2.0 ** -9 and numbers[8] == 2.0 ** -6
    x = torch.zeros(3, 40)
    x[0, :4] = torch.tensor([448.0, 1.0625, 1.1875, -2.0 ** -10])    # at scale 1: a tie to 1.0, one to 1.25, one to -0
    x[1, 0], x[1, 33] = 449.0, 2.0 ** -126
    codes, scales = R.pack(x)
    assert codes[0, :4].tolist() == [126, 56, 58, 128] and scales[0].tolist() == [127, 0]
    assert scales[1].tolist() == [128, 0] and scales[2].tolist() == [0, 0]
    back = R.unpack(codes, scales, 40)
    assert back[0, :4].tolist() == [448.0, 1.0, 1.25, 0.0] and back[1, 0] == 448.0 and back[1, 33] == 2.0 ** -126
    assert R.pack(torch.tensor([[INF, 3.0, NAN]]))[0][0, :3].tolist() == [127, 124, 127] and R.pack(torch.tensor([[INF, 3.0, NAN]]))[1] == 120


def test_frequencies_are_the_formulas():
    pytest.importorskip("torch")
    from mixed_precision_optimizer_bf16_gb300 import train_ops as ops
    import tuning_reference as R
    for how in (dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0), dict(scaling="yarn", factor=16.0, original_length=4096),
                dict(scaling="yarn", factor=1.0), dict(base=500000.0)):
        full = dict(base=10000.0, scaling=None, factor=1.0, original_length=2048, slow=1.0, fast=32.0)
        full.update(how)
        table, address, scale = ops._frequencies(64, *full.values())
        want, length = R.frequencies(64, **how)
        assert address == ctypes.addressof(table) and scale == length
        assert all(math.isclose(a, b, rel_tol=1e-14) for a, b in zip(table, want)) and len(table) == 32
    for bad in ((63, 1e4, None, 1.0, 1, 1, 2), (0, 1e4, None, 1.0, 1, 1, 2), (2, 1e4, "ntk", 2.0, 1, 1, 2), (64, 0.0, None, 1.0, 1, 1, 2),
                (64, 1e4, "linear", -1.0, 1, 1, 2), (64, 1e4, "other", 1.0, 1, 1, 2), (64, 1e4, "yarn", 2.0, 0, 1, 2), (64, 1e4, "yarn", 2.0, 1, 2, 2)):
        with pytest.raises(ValueError):
            ops._frequencies(*bad)


def test_host_tensors_are_refused():
    torch = pytest.importorskip("torch")
    from mixed_precision_optimizer_bf16_gb300 import train_ops as ops
    z, n = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    v, u = torch.zeros(4), torch.zeros(4, 32, dtype=torch.uint8)
    for call in (lambda: ops.token_logp_forward(z, n), lambda: ops.token_logp(z, n), lambda: ops.token_logp_backward(z, n, torch.zeros(4, 4)),
                 lambda: ops.policy_forward(z, n, v), lambda: ops.policy_loss(z, n, v), lambda: ops.policy_loss_grad(z, n, v),
                 lambda: ops.preference_forward(z, n, torch.zeros(3, dtype=torch.int32)), lambda: ops.preference_loss(z, n, n[:3]),
                 lambda: ops.pack8(z), lambda: ops.unpack8(u, u[:, :1], 32), lambda: ops.glu8_forward(z), lambda: ops.glu8(z, z),
                 lambda: ops.glu8_backward(z, u[None], u[None, :, :1]), lambda: ops.rotary_forward(z[:, None]), lambda: ops.rotary(z[:, None], z[:, None]),
                 lambda: ops.rotary_backward(z[:, None])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
