"""Refusals of the operators over pages and of the head norms: C entry points
(each returns before any CUDA call) and Python calls, without a GPU."""
import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

P = ctypes.c_void_p
FAKE, ODD = P(0x1000), P(0x1002)  # never dereferenced
OK, INVALID, ALIGN, SHAPE = 0, 1, 2, 3
BF16, INT, LONG, DOUBLE = torch.bfloat16, torch.int32, torch.int64, torch.float64


@pytest.fixture(scope="module")
def w():
    from w8a8_int8_linear_gb300 import build as b
    b.build()
    import w8a8_int8_linear_gb300 as w
    return w


@pytest.fixture(scope="module")
def L(w):
    return w.lib()


def paged(L, Q=FAKE, K=FAKE, V=FAKE, O=FAKE, lse=None, cu_q=None, table=FAKE, lens=FAKE, dtype=0, batch=1, Tq=4, most=0,
          pages=9, page_size=16, max_pages=3, table_stride=3, Hq=4, Hk=2, D=64,
          strides=(256, 64, 2048, 128, 64, 2048, 128, 64, 256, 64), scale=0.125, causal=1, ws=FAKE, ws_bytes=1 << 30):
    return L.w8a8_paged_attention(Q, K, V, O, lse, cu_q, table, lens, dtype, batch, Tq, most, pages, page_size, max_pages,
                                  table_stride, Hq, Hk, D, *strides, scale, causal, ws, ws_bytes, None)


def test_paged_attention(L):
    for kw in (dict(dtype=2), dict(dtype=-1), dict(batch=-1), dict(Tq=-1), dict(most=-1), dict(pages=-1),
               dict(page_size=0), dict(page_size=-16), dict(max_pages=-1), dict(table_stride=-1), dict(Hq=0), dict(Hk=0),
               dict(D=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(Q=None), dict(K=None), dict(V=None), dict(O=None), dict(table=None), dict(lens=None)):
        assert paged(L, **kw) == INVALID, kw
    for kw in (dict(D=12), dict(D=136), dict(Hq=5), dict(batch=3), dict(Tq=1 << 31), dict(page_size=12),
               dict(page_size=(1 << 20) + 8), dict(page_size=1 << 16, max_pages=1 << 15), dict(page_size=1024, max_pages=(1 << 21) - 1), dict(pages=1 << 31),
               dict(Hq=70000, Hk=1), dict(batch=1 << 31), dict(table_stride=1 << 31)):
        assert paged(L, **kw) == SHAPE, kw
    for i in range(10):
        for wrong in (4, 0, -8, 1 << 39):
            s = [256, 64, 2048, 128, 64, 2048, 128, 64, 256, 64]
            s[i] = s[i] + 4 if wrong == 4 else wrong
            assert paged(L, strides=s) == ALIGN, (i, wrong)
    for kw in (dict(Q=ODD), dict(K=ODD), dict(V=ODD), dict(O=ODD), dict(lse=ODD), dict(cu_q=ODD), dict(table=ODD),
               dict(lens=ODD)):
        assert paged(L, **kw) == ALIGN, kw
    assert paged(L, Tq=0, Q=None, O=None) == OK
    assert paged(L, batch=0) == OK


def norm(L, Q=FAKE, K=FAKE, Qo=FAKE, Ko=FAKE, dtype=0, T=4, Hq=4, Hk=2, D=64, rot=32,
         strides=(256, 64, 128, 64, 256, 64, 128, 64), qg=FAKE, qgs=0, kg=FAKE, kgs=64, eps=1e-6, kind=0, pos=FAKE,
         freqs=FAKE, amp=1.0, layout=0):
    return L.w8a8_qk_norm_rotary(Q, K, Qo, Ko, dtype, T, Hq, Hk, D, rot, *strides, qg, qgs, kg, kgs, eps, kind, pos, freqs,
                                 amp, layout, None)


APPEND = (256, 64, 128, 64, 128, 64, 256, 64, 2048, 128, 64, 2048, 128, 64)


def append(L, Q=FAKE, K=FAKE, V=FAKE, Qo=FAKE, Kc=FAKE, Vc=FAKE, dtype=0, T=4, Hq=4, Hk=2, D=64, rot=32, rows=160,
           page_size=16, strides=APPEND, qg=None, qgs=0, kg=None, kgs=0, eps=1e-6, kind=0, pos=FAKE, slots=FAKE,
           freqs=FAKE, amp=1.0, layout=0):
    return L.w8a8_qk_norm_rotary_append(Q, K, V, Qo, Kc, Vc, dtype, T, Hq, Hk, D, rot, rows, page_size, *strides, qg, qgs,
                                        kg, kgs, eps, kind, pos, slots, freqs, amp, layout, None)


def test_norm_rotary(L):
    both = [dict(dtype=2), dict(layout=2), dict(T=-1), dict(D=0), dict(rot=0), dict(amp=float("nan")), dict(kind=2),
            dict(kind=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(qgs=-8), dict(kgs=-8), dict(pos=None),
            dict(freqs=None), dict(Q=None), dict(K=None), dict(Qo=None)]
    for f, more in ((norm, [dict(Hq=-1), dict(Hk=-1), dict(Ko=None)]),
                    (append, [dict(Hk=0), dict(rows=-1), dict(page_size=-1), dict(slots=None), dict(V=None),
                              dict(Kc=None), dict(Vc=None)])):
        for kw in both + more:
            assert f(L, **kw) == INVALID, kw
        for kw in (dict(D=60), dict(D=264), dict(rot=24), dict(rot=80), dict(T=1 << 31), dict(Hq=70000)):
            assert f(L, **kw) == SHAPE, kw
        for kw in (dict(Q=ODD), dict(K=ODD), dict(Qo=ODD), dict(pos=ODD), dict(freqs=ODD), dict(qg=ODD), dict(kg=ODD),
                   dict(qgs=4), dict(kgs=4)):
            assert f(L, **kw) == ALIGN, kw
        default = (256, 64, 128, 64, 256, 64, 128, 64) if f is norm else APPEND
        for i in range(len(default)):
            s = list(default)
            s[i] += 2
            assert f(L, strides=s) == ALIGN, i
        assert f(L, T=0) == OK
    for i in range(4, 8):  # an output's rows on one another
        s = [256, 64, 128, 64, 256, 64, 128, 64]
        s[i] = 0
        assert norm(L, strides=s) == INVALID, i
    for i in range(6, 14):
        s = list(APPEND)
        s[i] = 0
        assert append(L, strides=s) == INVALID, i
    assert append(L, page_size=1 << 31) == SHAPE
    assert norm(L, Hq=0, Hk=0) == OK


def caches_of(n, ptr=0x1000, stride=4096):
    return (P * n)(*[ptr] * n), (ctypes.c_int64 * n)(*[stride] * n)


def copy(L, n_caches=2, base=None, strides=None, pages=5, page_bytes=4096, src=FAKE, dst=FAKE, n=3, **kw):
    c, s = caches_of(max(n_caches, 1), **kw)
    return L.w8a8_copy_pages(c if base is None else base, s if strides is None else strides, n_caches, pages, page_bytes,
                             src, dst, n, None)


def fork(L, n_caches=2, pages=5, page_bytes=4096, page_size=16, table=FAKE, rows=4, max_pages=3, table_stride=3,
         lens=FAKE, src=FAKE, dst=FAKE, new=FAKE, n=2, **kw):
    c, s = caches_of(max(n_caches, 1), **kw)
    return L.w8a8_fork_sequences(c, s, n_caches, pages, page_bytes, page_size, table, rows, max_pages, table_stride, lens,
                                 src, dst, new, n, None)


def test_pages(L):
    for f in (copy, fork):
        for kw in (dict(n=-1), dict(n_caches=-1), dict(pages=-1), dict(page_bytes=0), dict(src=None), dict(dst=None),
                   dict(ptr=None), dict(stride=4080)):
            assert f(L, **kw) == INVALID, kw
        for kw in (dict(pages=1 << 31), dict(page_bytes=(1 << 32) + 16)):
            assert f(L, **kw) == SHAPE, kw
        for kw in (dict(src=ODD), dict(dst=ODD), dict(ptr=0x1008), dict(stride=4100), dict(page_bytes=4088)):
            assert f(L, **kw) == ALIGN, kw
        assert f(L, n=0) == OK and f(L, n_caches=0) == OK and f(L, pages=0) == OK
    assert L.w8a8_copy_pages(None, None, 1, 5, 4096, FAKE, FAKE, 3, None) == INVALID
    for kw in (dict(rows=-1), dict(max_pages=-1), dict(page_size=0), dict(table_stride=-1), dict(table_stride=2),
               dict(table=None), dict(lens=None), dict(new=None)):
        assert fork(L, **kw) == INVALID, kw
    for kw in (dict(rows=1 << 31), dict(page_size=1 << 20, max_pages=1 << 12), dict(table_stride=1 << 31)):
        assert fork(L, **kw) == SHAPE, kw
    for kw in (dict(table=ODD), dict(lens=ODD), dict(new=ODD)):
        assert fork(L, **kw) == ALIGN, kw


X = torch.zeros(4, 2, 64, dtype=BF16)


@pytest.mark.parametrize("error,match,call", [
    (TypeError, "Q must be a torch.Tensor", lambda w: w.paged_attention([1], X, X, X, X)),
    (ValueError, "Q must be a CUDA tensor", lambda w: w.paged_attention(X, X, X, X, X)),
    (TypeError, "unexpected keyword", lambda w: w.paged_attention(X, X, X, X, X, window=3)),
    (ValueError, "Q must be a CUDA tensor", lambda w: w.qk_norm_rotary(X, X, X, X)),
    (ValueError, "layout must be 'half' or 'interleaved'", lambda w: w.qk_norm_rotary(X, X, X, X, layout="both")),
    (TypeError, "Q must be a torch.Tensor", lambda w: w.qk_norm_rotary_append(None, X, X, X, X, X, X, X)),
    (TypeError, "caches must be a list", lambda w: w.copy_pages(X, X, X)),
    (ValueError, "caches must hold a tensor", lambda w: w.copy_pages([], X, X)),
    (TypeError, r"caches\[1\] must be a torch.Tensor|caches\[0\] must be", lambda w: w.copy_pages([None], X, X)),
    (ValueError, r"caches\[0\] must be a CUDA tensor", lambda w: w.copy_pages([X], X, X)),
    (ValueError, r"caches\[0\] must be a CUDA tensor", lambda w: w.fork_sequences((X,), X, X, X, X, X, 16)),
])
def test_tensors_that_are_refused(w, error, match, call):
    with pytest.raises(error, match=match):
        call(w)


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake tensors of any GPU need a machine without one")
HEADS, PAGES = ((4, 2, 64), BF16), ((9, 16, 2, 64), BF16)
CALLS = {
    "paged_attention": dict(Q=HEADS, k_pages=PAGES, v_pages=PAGES, page_table=((2, 3), INT), k_lens=((2,), INT),
                            cu_q=((3,), INT), out=HEADS, workspace=((1 << 26,), torch.uint8)),
    "qk_norm_rotary": dict(Q=HEADS, K=HEADS, positions=((4,), LONG), freqs=((16,), DOUBLE), q_gamma=((64,), BF16),
                           k_gamma=((2, 64), BF16), q_out=HEADS, k_out=HEADS),
    "qk_norm_rotary_append": dict(Q=HEADS, K=HEADS, V=HEADS, positions=((4,), LONG), freqs=((16,), DOUBLE),
                                  k_cache=PAGES, v_cache=PAGES, slots=((4,), LONG), q_gamma=((64,), BF16),
                                  k_gamma=((64,), BF16), q_out=HEADS),
    "fork_sequences": dict(caches=PAGES, page_table=((4, 3), INT), k_lens=((4,), INT), src=((2,), INT), dst=((2,), INT),
                           new_pages=((2,), INT)),
    "copy_pages": dict(caches=PAGES, src=((2,), INT), dst=((2,), INT)),
}


def on(device, shape, dtype=BF16):
    with FakeTensorMode():
        return torch.empty(shape, dtype=dtype, device=device)


def arguments(call, other=None, **wrong):
    args = {n: on("cuda:1" if n == other else "cuda:0", *wrong.get(n, spec)) for n, spec in CALLS[call].items()}
    if "caches" in args:
        args["caches"] = [args["caches"]] * 2
    if call == "fork_sequences":
        args["page_size"] = 16
    return args


@needs_no_gpu
@pytest.mark.parametrize("call,name", [(c, n) for c, args in CALLS.items() for n in list(args)[1:]])
def test_another_gpu(w, call, name):
    first = next(iter(CALLS[call])).replace("caches", r"caches\[0\]")
    with pytest.raises(ValueError, match=f"{name} is on cuda:1, {first} on cuda:0"):
        getattr(w, call)(**arguments(call, name))


@needs_no_gpu
@pytest.mark.parametrize("call,name", [
    ("paged_attention", "out"), ("qk_norm_rotary", "q_out"), ("qk_norm_rotary", "k_out"),
    ("qk_norm_rotary_append", "k_cache"), ("qk_norm_rotary_append", "v_cache"), ("qk_norm_rotary_append", "q_out"),
    ("fork_sequences", "caches"), ("copy_pages", "caches")])
def test_written_tensors_that_require_a_gradient(w, call, name):
    args = arguments(call)
    (args[name][0] if name == "caches" else args[name]).requires_grad_()
    with pytest.raises(ValueError, match="requires a gradient"):
        getattr(w, call)(**args)


@needs_no_gpu
@pytest.mark.parametrize("call,name,spec,error,match", [
    ("paged_attention", "k_pages", ((9, 16, 2, 64), torch.float16), TypeError, "k_pages must be torch.bfloat16"),
    ("paged_attention", "k_pages", ((9, 2, 64), BF16), ValueError, r"k_pages must be \[pages, page_size, KV heads, dim\]"),
    ("paged_attention", "v_pages", ((9, 16, 1, 64), BF16), ValueError, "k_pages and v_pages must be"),
    ("paged_attention", "page_table", ((2, 3), LONG), TypeError, "page_table must be a torch.int32 tensor"),
    ("paged_attention", "page_table", ((6,), INT), ValueError, "page_table must be a CUDA tensor"),
    ("paged_attention", "k_lens", ((3,), INT), ValueError, "k_lens must be a dense CUDA tensor of 2 values"),
    ("paged_attention", "cu_q", ((2,), INT), ValueError, "cu_q must be a dense CUDA tensor of 3 values"),
    ("qk_norm_rotary", "q_gamma", ((64,), torch.float32), TypeError, "q_gamma must be torch.bfloat16"),
    ("qk_norm_rotary", "k_gamma", ((3, 64), BF16), ValueError, r"k_gamma must be a CUDA tensor \[dim\] or \[heads, dim\]"),
    ("qk_norm_rotary", "q_gamma", ((32,), BF16), ValueError, "q_gamma must be a CUDA tensor"),
    ("qk_norm_rotary_append", "k_cache", ((16, 2, 64), BF16), ValueError, "both caches"),
    ("qk_norm_rotary_append", "k_cache", ((2, 64), BF16), ValueError, r"or \[rows, KV heads, dim\]"),
    ("qk_norm_rotary_append", "slots", ((4,), INT), TypeError, "slots must be a torch.int64 tensor"),
    ("fork_sequences", "dst", ((3,), INT), ValueError, "dst must be a dense CUDA tensor of 2 values"),
    ("fork_sequences", "new_pages", ((2,), LONG), TypeError, "new_pages must be a torch.int32 tensor"),
    ("copy_pages", "src", ((2,), LONG), TypeError, "src must be a torch.int32 tensor"),
    ("copy_pages", "caches", ((9,), BF16), ValueError, r"caches\[0\] must be \[pages, ...\]"),
])
def test_shapes_and_types(w, call, name, spec, error, match):
    with pytest.raises(error, match=match):
        getattr(w, call)(**arguments(call, **{name: spec}))


@needs_no_gpu
def test_caches_of_several_kinds(w):
    args = arguments("copy_pages")
    a = args["caches"][0]
    for b, match in ((on("cuda:0", (8, 16, 2, 64)), "the same pages"), (on("cuda:0", (9, 16, 2, 32)), "the same pages"),
                     (on("cuda:1", (9, 16, 2, 64)), r"caches\[1\] is on cuda:1"),
                     (on("cuda:0", (9, 16, 2, 128))[..., :64], "dense pages")):
        with pytest.raises(ValueError, match=match):
            w.copy_pages([a, b], args["src"], args["dst"])
    with pytest.raises(ValueError, match="k_gamma and k_out need K"):
        w.qk_norm_rotary(**{**arguments("qk_norm_rotary"), "K": None})
