"""The 4-bit rows and the low-bit cache without a GPU: the headers' exports, the refusals of the
C calls and of the binding, the slot arithmetic on the host, and the float64 definitions."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

from oracle import gptq_ref as o
from oracle import lowbit_ref as L
from post_weight_quantization_20_b200 import gptq as G
from post_weight_quantization_20_b200 import kv_cache as KV
from post_weight_quantization_20_b200 import mx as MX

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INCLUDE = os.path.join(ROOT, "include")
no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="passes fake device pointers; only run without a GPU")
FAKE = ctypes.c_void_p(4096)
INVALID, UNSUPPORTED, OK = G.GPTQ_ERR_INVALID_ARG, G.GPTQ_ERR_UNSUPPORTED, G.GPTQ_OK


@pytest.mark.parametrize("header,module", [("gptq_mx.h", MX), ("gptq_cache.h", KV)])
def test_header_declares_what_the_binding_exports(header, module):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(INCLUDE, header)).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(gptq_(?:mx|cache)_[a-z_]+)\s*\(", src)))
    assert names == sorted(module.EXPORTS)
    lib = module.load_library()
    for n in names:
        assert hasattr(lib, n), n


def test_headers_compile_as_c99(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "t.c"
    # and the structures lie in memory as the binding packs them
    src.write_text('#include <stddef.h>\n#include "gptq_mx.h"\n#include "gptq_cache.h"\n'
                   "int main(void) { gptq_cache_config c = {GPTQ_CACHE_GRID, 8, 0, 0};\n"
                   f"  if (sizeof(gptq_cache) != {KV._CACHE.size} || offsetof(gptq_cache, dim) != 56 ||\n"
                   f"      sizeof(gptq_cache_rows) != {KV._ROWS.size} || offsetof(gptq_cache_rows, cu) != 24)\n"
                   "    return 2;\n"
                   "  return gptq_mx_scale_bytes(1, 1) == 512 && gptq_cache_words(&c, 64) == 16 ? 0 : 1; }\n")
    libdir = os.path.dirname(G.LIB_PATH)
    MX.load_library()
    exe = tmp_path / "t"
    r = subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", INCLUDE,
                        str(src), "-o", str(exe), "-L", libdir, "-lgptq", f"-Wl,-rpath,{libdir}"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert subprocess.run([str(exe)], timeout=120).returncode == 0


# ------------------------------------------------------------------ refusals of the C calls
def test_mx_sizes():
    assert MX.gptq_mx_scale_bytes(1, 1) == 512
    assert MX.gptq_mx_scale_bytes(129, 129) == 4 * 512
    assert MX.gptq_mx_scale_bytes(0, 5) == 0 and MX.gptq_mx_scale_bytes(-1, 5) == 0
    assert MX.gptq_mx_scale_bytes(5, 0) == 0
    for r, c in ((1, 1), (128, 128), (129, 4097), (7, 32)):
        shape = MX.mx_scale_shape(r, c)
        assert int(np.prod(shape)) == MX.gptq_mx_scale_bytes(r, c)
    assert [MX.mx_words(c) for c in (1, 32, 33)] == [4, 4, 8]


@no_gpu
def test_mx_quantize_and_dequantize_refuse_bad_arguments():
    lib = MX.load_library()
    odd = ctypes.c_void_p(4104)
    for args, want in (((FAKE, 7, 4, 32, 32, FAKE, FAKE), INVALID),        # dtype
                       ((FAKE, 1, -1, 32, 32, FAKE, FAKE), INVALID),
                       ((FAKE, 1, 4, 0, 32, FAKE, FAKE), INVALID),
                       ((FAKE, 1, 4, 32, 31, FAKE, FAKE), INVALID),        # ldx < cols
                       ((None, 1, 4, 32, 32, FAKE, FAKE), INVALID),
                       ((FAKE, 1, 4, 32, 32, None, FAKE), INVALID),
                       ((FAKE, 1, 4, 32, 32, odd, FAKE), INVALID),         # codes not 16-byte aligned
                       ((FAKE, 1, 4, 32, 32, FAKE, odd), INVALID),
                       ((FAKE, 1, 2 ** 31, 32, 32, FAKE, FAKE), INVALID),
                       ((FAKE, 1, 2 ** 31 - 1, 2 ** 30 - 1, 2 ** 30, FAKE, FAKE), INVALID),   # grid
                       ((None, 1, 0, 32, 32, None, None), OK)):            # no rows: a no-op
        assert lib.gptq_mx_quantize(*args, None, None) == want, args
        X, dt, r, c, ld, codes, scales = args
        assert lib.gptq_mx_dequantize(codes, scales, r, c, X, dt, ld, None) == want, args


@no_gpu
def test_mx_matmul_refuses_bad_arguments():
    f = MX.load_library().gptq_mx_matmul
    ok = dict(xc=FAKE, xs=FAKE, M=2, wc=FAKE, ws=FAKE, R=8, C=64, Y=FAKE, dt=0, ld=8)

    def call(**over):
        a = dict(ok, **over)
        return f(a["xc"], a["xs"], a["M"], a["wc"], a["ws"], a["R"], a["C"], a["Y"], a["dt"],
                 a["ld"], None, None)

    odd = ctypes.c_void_p(4104)
    for over in (dict(xc=None), dict(xs=None), dict(wc=None), dict(ws=None), dict(Y=None),
                 dict(M=-1), dict(R=-1), dict(C=0), dict(dt=3), dict(ld=7), dict(xc=odd),
                 dict(xs=odd), dict(wc=odd), dict(ws=odd), dict(M=2 ** 31)):
        assert call(**over) == INVALID, over
    for over in (dict(M=0, xc=None, Y=None), dict(R=0, wc=None, ld=0)):
        assert call(**over) == OK, over


@no_gpu
def test_mx_matmul_refuses_sizes_past_its_index_arithmetic():
    f, top = MX.load_library().gptq_mx_matmul, 2 ** 31 - 1
    launched = (G.GPTQ_ERR_CUDA,)                        # past the checks: there is no GPU here

    def call(M, R):
        return f(FAKE, FAKE, M, FAKE, FAKE, R, 32, FAKE, 0, R, None, None)

    for M, R in ((1, top), (top, 1), (1, top - 254), (top - 254, 1), (100, top - 100),
                 (2 ** 23, 2 ** 22 * 8), (top - 255, top - 255)):
        assert call(M, R) == INVALID, (M, R)
    for M, R in ((1, top - 255), (top - 255, 1), (2 ** 22, 2 ** 22)):
        assert call(M, R) in launched, (M, R)


def test_give_up_stage_is_off_by_default_and_returned():
    assert MX.gptq_mx_debug_give_up(3) == -1
    assert MX.gptq_mx_debug_give_up(-7) == 3
    assert MX.gptq_mx_debug_give_up(-1) == -1


def _cache_args(cfg=None, **over):
    c = dict(k_codes=4096, k_grids=4096, v_codes=4096, v_grids=4096, pages=4, page_size=16,
             heads=2, dim=64)
    r = dict(table=4096, table_ld=4, width=4, cu=4096, start=4096, seqs=1)
    a = dict(K=FAKE, V=FAKE, dt=1, tokens=3)
    for k, v in over.items():
        next(d for d in (c, r, a) if k in d)[k] = v
    null = lambda d: [v or 0 for v in d.values()]  # noqa: E731
    return a, cfg or KV.make_cache_config("grid", 4, 32), KV._CACHE.pack(*null(c)), KV._ROWS.pack(*null(r))


def _cache_calls(cfg=None, **over):
    a, cfg, c, r = _cache_args(cfg, **over)
    lib, ref = KV.load_library(), ctypes.byref
    st = (128, 64, 128, 64)
    w = lib.gptq_cache_write(a["K"], a["V"], a["dt"], a["tokens"], *st, ref(cfg), c, r, None, None)
    d = lib.gptq_cache_read(ref(cfg), c, r, a["K"], a["V"], a["dt"], a["tokens"], *st, None, None)
    assert w == d
    return w


@no_gpu
def test_cache_calls_refuse_bad_arguments():
    for over in (dict(K=None), dict(V=None), dict(dt=4), dict(tokens=-1), dict(pages=-1),
                 dict(page_size=0), dict(heads=0), dict(dim=0), dict(width=-1), dict(table_ld=3),
                 dict(seqs=-1), dict(cu=None), dict(start=None), dict(table=None),
                 dict(k_codes=None), dict(v_grids=None), dict(k_codes=4104), dict(v_grids=4104)):
        assert _cache_calls(**over) == INVALID, over
    for cfg in (("grid", 3, 32, False), ("grid", 2, 32, False), ("mx", 8, 32, False), ("grid", 4, -1, False)):
        assert _cache_calls(KV.make_cache_config(*cfg)) == INVALID, cfg
    bad = KV.make_cache_config("grid", 4, 32)
    bad.kind = 2
    assert _cache_calls(bad) == INVALID
    assert _cache_calls(dim=60) == UNSUPPORTED                       # not a multiple of 8
    assert _cache_calls(KV.make_cache_config("grid", 4, 48)) == UNSUPPORTED
    assert _cache_calls(KV.make_cache_config("grid", 4, 0), dim=264) == UNSUPPORTED
    assert _cache_calls(KV.make_cache_config("mx", 4, 64)) == UNSUPPORTED
    assert _cache_calls(tokens=0, K=None) == OK                      # no-ops
    assert _cache_calls(seqs=0, cu=None) == OK


def test_cache_sizes():
    for kind, bits, g, dim, words, grid in (("grid", 4, 0, 80, 10, 8), ("grid", 8, 32, 80, 20, 24),
                                            ("grid", 4, 64, 128, 16, 16), ("mx", 4, 32, 80, 12, 3),
                                            ("mx", 4, 0, 64, 8, 2)):
        cfg = KV.make_cache_config(kind, bits, g)
        assert KV.gptq_cache_words(cfg, dim) == words == KV._words(cfg, dim)
        assert KV.gptq_cache_grid_bytes(cfg, dim) == grid
        shape, dt = KV._grid_shape(cfg, 1, 1, 1, dim)
        assert int(np.prod(shape)) * torch.empty((), dtype=dt).element_size() == grid
    assert KV.gptq_cache_words(KV.make_cache_config("grid", 4, 0), 264) == 0
    assert KV.gptq_cache_grid_bytes(KV.make_cache_config("grid", 5, 0), 64) == 0
    with pytest.raises(ValueError, match="kind"):
        KV.make_cache_config("fp8")
    with pytest.raises(G.GPTQError):
        KV.KVCache.alloc(KV.make_cache_config("grid", 4, 48), 1, 1, 1, 64, device="cpu")


# ------------------------------------------------------------------ refusals of the binding
def test_mx_binding_checks_its_tensors():
    X = torch.zeros(4, 100, dtype=torch.float16)
    codes, scales = torch.zeros(4, 16, dtype=torch.int32), torch.zeros(1, 1, 32, 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensors"):          # everything else fits
        MX.gptq_mx_quantize(X, codes, scales)
    with pytest.raises(ValueError, match="device tensors"):
        MX.gptq_mx_dequantize(codes, scales, X)
    for args, word in (((X.double(), codes, scales), "X"), ((X.t(), codes, scales), "X"),
                       ((X[0], codes, scales), "X"), ((X, codes[:, :-1], scales), "codes"),
                       ((X, codes.long(), scales), "codes"), ((X, codes, scales[0]), "scales"),
                       ((X, codes, scales.int()), "scales"), ((X[:1].expand(4, 100), codes, scales), "X")):
        with pytest.raises(ValueError, match=word):
            MX.gptq_mx_quantize(*args)
    with pytest.raises(ValueError, match="status"):
        MX.gptq_mx_quantize(X, codes, scales, torch.zeros(1))
    Y = torch.zeros(4, 4)
    with pytest.raises(ValueError, match="device tensors"):
        MX.gptq_mx_matmul(codes, scales, codes, scales, 100, Y)
    for args, word in (((codes, scales, codes, scales, 100, Y[:3]), "x_codes"),
                       ((codes, scales, codes[:3], scales, 100, Y), "w_codes"),
                       ((codes, scales, codes, scales, 140, Y), "x_codes"),
                       ((codes, scales, codes, scales.int(), 100, Y), "w_scales"),
                       ((codes, scales, codes, scales, 100, Y.double()), "Y")):
        with pytest.raises(ValueError, match=word):
            MX.gptq_mx_matmul(*args)
    a = MX.MXMatrix(codes, scales, 4, 100)
    with pytest.raises(ValueError, match="cols"):
        MX.mx_matmul(a, MX.MXMatrix(codes, scales, 4, 101))


def test_cache_binding_checks_its_tensors():
    cfg = KV.make_cache_config("grid", 4, 32)
    K = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    codes = torch.zeros(5, 16, 2, 8, dtype=torch.int32)
    grids = torch.zeros(5, 16, 2, 2, 2)
    table = torch.zeros(1, 4, dtype=torch.int32)
    cu, start = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    ok = dict(K=K, V=K, cfg=cfg, k_codes=codes, k_grids=grids, v_codes=codes, v_grids=grids,
              table=table, cu=cu, start=start)
    for f in (KV.gptq_cache_write, KV.gptq_cache_read):
        with pytest.raises(ValueError, match="device tensors"):
            f(**ok)
        for over, word in ((dict(K=K[0]), "K"), (dict(K=K.double()), "K"), (dict(V=K[:2]), "V"),
                           (dict(V=K.half()), "V"), (dict(K=K.transpose(1, 2)), "K"),
                           (dict(k_codes=codes[0]), "k_codes"), (dict(v_codes=codes[..., :7]), "v_codes"),
                           (dict(k_grids=grids[..., 0]), "k_grids"), (dict(v_grids=grids.double()), "v_grids"),
                           (dict(table=table.long()), "table"), (dict(table=table[0]), "table"),
                           (dict(cu=cu[:1]), "cu"), (dict(start=start.float()), "start"),
                           (dict(cfg=KV.make_cache_config("mx")), "k_grids"),
                           (dict(cfg=KV.make_cache_config("grid", 8, 32)), "k_codes")):
            with pytest.raises(ValueError, match=word):
                f(**dict(ok, **over))
    with pytest.raises(ValueError, match="overlap"):                 # a read writes K and V
        KV.gptq_cache_read(**dict(ok, K=K[:1].expand(3, 2, 64)))


# ------------------------------------------------------------------ slots on the host
def test_slot_arithmetic_on_the_host(tmp_path):
    # the device code's own function, compiled for the host, on ragged, empty, padded, negative
    # and out-of-range rows; the arrays are exactly as long as the call may read
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src = tmp_path / "slots.cc"
    src.write_text('#include "kv_slots.h"\n'
                   'extern "C" void slots(const int32_t* table, int64_t ld, int64_t width, int64_t pages,\n'
                   '    const int32_t* cu, const int32_t* start, int seqs, int page, int64_t n, int64_t* out) {\n'
                   '  const gptq::RowMap m = {table, ld, width, pages, cu, start, seqs, page};\n'
                   '  for (int64_t t = 0; t < n; ++t) out[t] = gptq::slot_of(m, t); }\n')
    so = tmp_path / "slots.so"
    subprocess.run([cxx, "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "post_weight_quantization_20_b200", "csrc"), str(src), "-o",
                    str(so)], check=True)
    f = ctypes.CDLL(str(so)).slots
    rng = np.random.default_rng(3)
    for trial in range(200):
        S, page, width, pages = (int(v) for v in rng.integers(1, [9, 20, 5, 30]))
        new = rng.integers(0, 12, S)
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        start = rng.integers(-3, 40, S).astype(np.int32)
        table = rng.integers(-2, pages + 2, (S, width)).astype(np.int32)
        n = int(cu[-1]) + 3
        out = np.empty(n, np.int64)
        i64 = ctypes.c_int64
        f(table.ctypes.data_as(ctypes.c_void_p), i64(width), i64(width), i64(pages),
          cu.ctypes.data_as(ctypes.c_void_p), start.ctypes.data_as(ctypes.c_void_p), S, page,
          i64(n), out.ctypes.data_as(ctypes.c_void_p))
        np.testing.assert_array_equal(out, L.slots(n, table, cu, start, page, pages))
    # far positions: the products stay in 64 bits
    big = 2 ** 31 - 1
    table = np.array([[0] * 3 + [big - 1]], dtype=np.int32)
    cu, start = np.array([0, 2], np.int32), np.array([4 * 2 ** 20 - 2], np.int32)
    out = np.empty(3, np.int64)
    f(table.ctypes.data_as(ctypes.c_void_p), i64(4), i64(4), i64(big),
      cu.ctypes.data_as(ctypes.c_void_p), start.ctypes.data_as(ctypes.c_void_p), 1, 2 ** 20, i64(3),
      out.ctypes.data_as(ctypes.c_void_p))
    assert out.tolist() == [(big - 1) * 2 ** 20 + 2 ** 20 - 2, (big - 1) * 2 ** 20 + 2 ** 20 - 1, -1]


# ------------------------------------------------------------------ accumulators on the host
def test_accumulators_are_all_handed_back_before_a_pair_parts(tmp_path):
    # The device code's own turn-taking, compiled for the host, on a model of the barriers: the
    # waits before each use pass as soon as the use before it was handed back and no sooner, and
    # the waits at the end do not pass while any arrival of the last uses is outstanding.
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src = tmp_path / "ring.cc"
    src.write_text('#include "acc_ring.h"\n'
                   "// passes of a barrier with `done` completed phases for a wait on `parity`\n"
                   "static bool passes(int done, uint32_t parity) { return uint32_t(done & 1) != parity; }\n"
                   'extern "C" int run(int accs, int tiles) {\n'
                   "  gptq::AccRing mma(accs), epi(accs);\n"
                   "  int uses[2] = {0, 0}, back[2] = {0, 0};\n"
                   "  for (int t = 0; t < tiles; ++t) {\n"
                   "    if (mma.at != t % accs) return 1;\n"
                   "    // as late as it may be: handed back only when this use needs it\n"
                   "    while (back[mma.at] < uses[mma.at]) {\n"
                   "      if (passes(back[mma.at], mma.phase ^ 1u)) return 2;\n"
                   "      if (epi.at != mma.at || epi.phase != (back[epi.at] & 1u)) return 3;\n"
                   "      ++back[epi.at];\n"
                   "      epi.next();\n"
                   "    }\n"
                   "    if (!passes(back[mma.at], mma.phase ^ 1u)) return 4;\n"
                   "    ++uses[mma.at];\n"
                   "    mma.next();\n"
                   "  }\n"
                   "  for (int i = 0; i < accs; ++i) {\n"
                   "    if (uses[i] - back[i] > 1) return 5;\n"
                   "    if (back[i] < uses[i] && passes(back[i], mma.last(i))) return 6;   // outstanding\n"
                   "    if (!passes(uses[i], mma.last(i))) return 7;                       // landed, or never used\n"
                   "  }\n"
                   "  return 0; }\n")
    so = tmp_path / "ring.so"
    subprocess.run([cxx, "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "post_weight_quantization_20_b200", "csrc"), str(src), "-o",
                    str(so)], check=True)
    run = ctypes.CDLL(str(so)).run
    for accs in (1, 2):
        for tiles in range(12):
            assert run(accs, tiles) == 0, (accs, tiles)
    # and the product's MMA warp makes those waits
    src = open(os.path.join(ROOT, "post_weight_quantization_20_b200", "csrc", "mx_matmul.cu")).read()
    assert "wait(acc_empty + i, ring.last(i), true)" in src


def test_epilogues_wait_as_whole_warps():
    # tcgen05.ld is .aligned: the wait before it must give all lanes of a warp one answer
    csrc = os.path.join(ROOT, "post_weight_quantization_20_b200", "csrc")
    votes = {"mbar_wait_warp", "mbar_wait_pair_warp", "wait"}
    found = 0
    for name in ("mx_matmul.cu", "gemm_tc.cu", "hessian_tc.cu"):
        src = open(os.path.join(csrc, name)).read()
        calls = set(re.findall(r"(\w*wait\w*)\(acc_full\b", src))
        assert calls and calls <= votes, (name, calls)
        found += len(re.findall(r"wait\w*\(acc_full\b", src))
    assert found == 5
    assert "return tc::mbar_wait_pair_warp(bar," in open(os.path.join(csrc, "mx_matmul.cu")).read()


def test_both_ctas_of_a_pair_see_the_end_of_an_abort():
    # the issuer's arrivals reach both CTAs of a pair; after a wait gave up, both wait for the last
    csrc = os.path.join(ROOT, "post_weight_quantization_20_b200", "csrc")
    for name, both in (("mx_matmul.cu", "both"), ("hessian_tc.cu", "0x3")):
        src = open(os.path.join(csrc, name)).read()
        assert set(re.findall(r"mma_commit_pair\([^,]+, ([^)]+)\)", src)) == {both}, name


# ------------------------------------------------------------------ the definitions
def test_mx_definition_on_hand_worked_blocks():
    x = np.zeros((4, 32))
    # top 6: scale 1; ties to the even code: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    x[0, :9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5]
    x[1, :3] = [7.9, -7.9, 3]                    # above 6 scales: saturates
    x[2, :2] = [2.0 ** -130, 2.0 ** -127]        # below the least scale: e = 0
    x[3, :2] = [np.inf, 1]
    c, e = L.mx_quantize(x)
    assert e[:, 0].tolist() == [127, 127, 0, 255]
    v = L.mx_values(c, e)
    assert v[0, :9].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -4]
    assert v[1, :3].tolist() == [6, -6, 3]
    assert v[2, :2].tolist() == [0.0, 2.0 ** -127]
    assert np.isnan(v[3]).all() and not c[3].any()


def test_mx_pack_is_the_bitstream_of_gptq_pack_and_tiles_are_a_permutation():
    rng = np.random.default_rng(0)
    c, e = L.mx_quantize(rng.standard_normal((3, 70)))
    w = o.pack(c.astype(np.int64), 4)
    assert w.shape == (3, MX.mx_words(70))
    assert [(int(w[1, j // 8]) >> (4 * (j % 8))) & 15 for j in range(96)] == c[1].tolist()
    nb = 9
    seen = {L.mx_scale_index(r, k, nb) for r in range(256) for k in range(12)}
    assert seen == set(range(2 * 3 * 512))
    assert L.mx_tile(e).reshape(MX.mx_scale_shape(3, 70))[0, 0, 2, 1] == e[2, 1]


def test_grid_definition_matches_the_weight_grid_and_its_edges():
    rng = np.random.default_rng(1)
    x = np.float32(rng.standard_normal((5, 64))).astype(np.float64)
    for bits, sym in ((4, False), (8, False), (4, True)):
        c, s, z = L.grid_quantize(x, bits, 32, sym)
        for g in range(2):                       # the grid of the weights' sweep
            sc, zo = o.grid(x[:, 32 * g:32 * g + 32], bits, sym)[:2]
            np.testing.assert_array_equal(np.float32(sc), s[:, g])
            np.testing.assert_array_equal(zo, z[:, g])
        err = np.abs(L.grid_values(c, s, z, 32) - x)
        assert np.all(err <= np.repeat(s, 32, 1) * (0.5 + 2.0 ** -10))
    edge = np.zeros((4, 8))
    edge[1, 3] = np.nan
    edge[2, :2] = [3e38, -3e38]                       # range overflows fp32
    edge[3, 0] = 2.0 ** -149                          # range underflows
    c, s, z = L.grid_quantize(edge, 4, 0, False)
    v = L.grid_values(c, s, z, 0)
    assert (v[0] == 0).all() and np.isnan(v[1]).all() and np.isnan(v[2]).all() and (v[3] == 0).all()


def test_calls_run_on_their_tensors_device_and_current_stream(monkeypatch):
    # tensors of a device that is not the current one: that device is made current for the
    # launch, and its own current stream is taken, not the other device's
    import contextlib
    seen = []

    @contextlib.contextmanager
    def device(d):
        seen.append(("enter", d))
        yield
        seen.append(("leave", d))

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 1000 + d, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    MX._call(lambda *a: seen.append(a) or 0, "f", 0, None, "x")
    assert seen == [("enter", 0), ("x", 1000), ("leave", 0)]
    seen.clear()
    MX._call(lambda *a: seen.append(a) or 0, "f", 1, None, "x")
    assert seen == [("x", 1001)]
    seen.clear()

    class Stream:
        cuda_stream = 77

    MX._call(lambda *a: seen.append(a) or 0, "f", 1, Stream(), "x")
    assert seen == [("x", 77)]
    with pytest.raises(G.GPTQError) as e:
        MX._call(lambda *a: G.GPTQ_ERR_UNSUPPORTED, "f", 1, None)
    assert e.value.code == G.GPTQ_ERR_UNSUPPORTED
