"""The entry points of gdn_attn.h reject bad arguments on the host before any
HIP call (so these run without a GPU), and their host layer runs clean under
AddressSanitizer and UndefinedBehaviorSanitizer."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import gated_deltanet_tree_gdn_amd as gdn
from gated_deltanet_tree_gdn_amd import attn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdn_attn.h")
FAKE = 0x10000  # never dereferenced: every call below fails before touching it


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdn.LIB_PATH):
        pytest.fail("libgdn_tree.so is not built: run __graft_entry__.build()")
    return attn.attn_library()


def status(code):
    return gdn.STATUS[code]


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(gdn_[a-z0-9_]+)\s*\(", text))
    assert names == set(attn.ATTN_EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


def cache(**kw):
    d = dict(k=FAKE, v=FAKE + 4096, k_scale=None, v_scale=None, n_pages=10, page_size=16, H_kv=2, d=128, dtype=0, reserved=0,
             k_page_stride=4096, k_row_stride=256, k_head_stride=128, v_page_stride=4096, v_row_stride=256, v_head_stride=128)
    d.update(kw)
    return attn.KvCacheStruct(**d)


def dims(**kw):
    d = dict(B=3, T=20, H_q=8, max_pages=40, scale=0.1, reserved=0, q_stride=1024, gate_stride=1024, gate_head_stride=128,
             table_stride=40)
    d.update(kw)
    return attn.AttnDims(**d)


KINDS = {"decode": ["q", "table", "length", "gate", "o", "seq_status", "workspace"],
         "prefill": ["q", "cu_seqlens", "table", "length", "gate", "o", "seq_status", "workspace"],
         "verify": ["q", "anc", "table", "length", "gate", "o", "seq_status", "workspace"]}


def need(lib, kind, d, c):
    return getattr(lib, f"gdn_attn_{kind}_workspace_bytes")(d, c)


def call(lib, kind, d, c, nbytes=None, **over):
    a = {n: FAKE + 256 * i for i, n in enumerate(KINDS[kind])}
    a.update(over)
    if nbytes is None:
        nbytes = need(lib, kind, d, c)
    return status(getattr(lib, f"gdn_attn_{kind}")(d, c, *(a[n] for n in KINDS[kind]), nbytes, None))


BAD_CACHE = [
    (dict(dtype=1), "GDN_ERR_DTYPE"), (dict(dtype=3), "GDN_ERR_DTYPE"), (dict(d=96), "GDN_ERR_SHAPE"), (dict(d=512), "GDN_ERR_SHAPE"),
    (dict(n_pages=0), "GDN_ERR_SHAPE"), (dict(page_size=0), "GDN_ERR_SHAPE"), (dict(page_size=24), "GDN_ERR_SHAPE"),
    (dict(page_size=131072), "GDN_ERR_SHAPE"), (dict(page_size=-16), "GDN_ERR_SHAPE"),
    (dict(n_pages=1 << 20, page_size=4096), "GDN_ERR_SHAPE"), (dict(H_kv=0), "GDN_ERR_SHAPE"), (dict(H_kv=65536), "GDN_ERR_SHAPE"),
    (dict(reserved=1), "GDN_ERR_SHAPE"), (dict(k_page_stride=-8), "GDN_ERR_SHAPE"), (dict(v_row_stride=1 << 41), "GDN_ERR_SHAPE"), (dict(k_row_stride=(1 << 24) + 8), "GDN_ERR_SHAPE"),
    (dict(k_row_stride=4), "GDN_ERR_ALIGN"), (dict(v_head_stride=130), "GDN_ERR_ALIGN"), (dict(dtype=2, k_head_stride=136), "GDN_ERR_ALIGN"),
    (dict(k=None), "GDN_ERR_NULL"), (dict(v=None), "GDN_ERR_NULL"), (dict(k=FAKE + 8), "GDN_ERR_ALIGN"), (dict(v=FAKE + 2), "GDN_ERR_ALIGN"),
    (dict(k_scale=FAKE + 2), "GDN_ERR_ALIGN"), (dict(v_scale=FAKE + 1), "GDN_ERR_ALIGN"),
]
BAD_DIMS = [
    (dict(B=-1), "GDN_ERR_SHAPE"), (dict(B=65536), "GDN_ERR_SHAPE"), (dict(H_q=0), "GDN_ERR_SHAPE"), (dict(H_q=7), "GDN_ERR_SHAPE"),
    (dict(max_pages=-1), "GDN_ERR_SHAPE"), (dict(max_pages=1 << 27), "GDN_ERR_SHAPE"), (dict(scale=-1.0), "GDN_ERR_SHAPE"),
    (dict(scale=float("nan")), "GDN_ERR_SHAPE"), (dict(scale=float("inf")), "GDN_ERR_SHAPE"), (dict(reserved=1), "GDN_ERR_SHAPE"),
    (dict(q_stride=-8), "GDN_ERR_SHAPE"), (dict(q_stride=1028), "GDN_ERR_ALIGN"), (dict(gate_stride=-1), "GDN_ERR_SHAPE"),
    (dict(gate_head_stride=-1), "GDN_ERR_SHAPE"), (dict(table_stride=-1), "GDN_ERR_SHAPE"), (dict(B=65535, H_q=1 << 16), "GDN_ERR_SHAPE"),
]


@pytest.mark.parametrize("kind", KINDS)
def test_attention_rejects_sizes(lib, kind):
    for kw, code in BAD_CACHE:
        assert call(lib, kind, dims(), cache(**kw), nbytes=1 << 40) == code, kw
        assert lib.gdn_last_error().decode()
        assert need(lib, kind, dims(), cache(**kw)) == 0
    for kw, code in BAD_DIMS:
        if kind != "decode" and kw.get("B") == 65535:
            kw = dict(kw, T=256) if kind == "verify" else dict(T=1 << 20, H_q=1 << 12)
        assert call(lib, kind, dims(**kw), cache(), nbytes=1 << 40) == code, kw
        assert need(lib, kind, dims(**kw), cache()) == 0
    if kind != "decode":
        assert call(lib, kind, dims(T=-1), cache(), nbytes=1 << 40) == "GDN_ERR_SHAPE"
    if kind == "verify":
        assert call(lib, kind, dims(T=257), cache(), nbytes=1 << 40) == "GDN_ERR_SHAPE"
    fn = getattr(lib, f"gdn_attn_{kind}")
    rest = [FAKE] * len(KINDS[kind])
    assert status(fn(None, cache(), *rest, 1 << 40, None)) == "GDN_ERR_NULL"
    assert status(fn(dims(), None, *rest, 1 << 40, None)) == "GDN_ERR_NULL"


def test_rows_are_numbered_in_32_bits(lib):
    """the last tile's 128 rows too"""
    most = (1 << 31) - 256
    for T in (most // 8 + 1, (1 << 28) - 1):
        assert call(lib, "prefill", dims(T=T, H_q=8), cache(), nbytes=1 << 40) == "GDN_ERR_SHAPE"
        assert need(lib, "prefill", dims(T=T, H_q=8), cache()) == 0
    assert need(lib, "prefill", dims(T=most // 8, H_q=8), cache()) > 0


@pytest.mark.parametrize("kind", KINDS)
def test_attention_rejects_pointers(lib, kind):
    odd = dict(q=8, cu_seqlens=2, anc=2, table=2, length=1, gate=1, o=8, seq_status=2)
    for name, shift in odd.items():
        if name in KINDS[kind]:
            assert call(lib, kind, dims(), cache(), **{name: FAKE + shift}) == "GDN_ERR_ALIGN", name
            if name not in ("gate", "seq_status"):
                assert call(lib, kind, dims(), cache(), **{name: None}) == "GDN_ERR_NULL", name
                assert name in lib.gdn_last_error().decode()
    assert call(lib, kind, dims(), cache(), o=FAKE, q=FAKE) == "GDN_ERR_SHAPE"
    n = need(lib, kind, dims(), cache())
    assert n > 0 and n % 256 == 0
    assert call(lib, kind, dims(), cache(), workspace=None) == "GDN_ERR_WORKSPACE"
    assert call(lib, kind, dims(), cache(), nbytes=n - 1) == "GDN_ERR_WORKSPACE"
    assert call(lib, kind, dims(), cache(), workspace=FAKE + 128) == "GDN_ERR_ALIGN"
    nothing = dict.fromkeys(KINDS[kind])
    assert call(lib, kind, dims(B=0), cache(), **nothing) == "GDN_OK"
    assert need(lib, kind, None, cache()) == need(lib, kind, dims(), None) == need(lib, kind, dims(B=0), cache()) == 0


def append_dims(**kw):
    d = dict(T=3, H_q=8, in_dtype=0, rot=64, interleaved=0, eps=1e-6, weight_offset=0.0, reserved=0, q_stride=1024,
             q_head_stride=128, k_stride=256, k_head_stride=128, v_stride=256, v_head_stride=128)
    d.update(kw)
    return attn.AppendDims(**d)


APPEND = ["q", "k", "v", "q_weight", "k_weight", "inv_freq", "position", "slot", "q_out"]


def append(lib, d, c, **over):
    a = {n: FAKE + 256 * i for i, n in enumerate(APPEND)}
    a.update(over)
    return status(lib.gdn_kv_append(d, c, *(a[n] for n in APPEND), None))


def test_append_rejects(lib):
    for kw, code in BAD_CACHE:
        assert append(lib, append_dims(), cache(**kw)) == code, kw
    for kw, code in [(dict(T=-1), "GDN_ERR_SHAPE"), (dict(H_q=-1), "GDN_ERR_SHAPE"), (dict(H_q=65536), "GDN_ERR_SHAPE"),
                     (dict(in_dtype=2), "GDN_ERR_DTYPE"), (dict(rot=-2), "GDN_ERR_SHAPE"), (dict(rot=33), "GDN_ERR_SHAPE"),
                     (dict(rot=130), "GDN_ERR_SHAPE"), (dict(interleaved=2), "GDN_ERR_SHAPE"), (dict(eps=-1.0), "GDN_ERR_SHAPE"),
                     (dict(eps=float("nan")), "GDN_ERR_SHAPE"), (dict(reserved=3), "GDN_ERR_SHAPE"),
                     *[(dict([(n, -1)]), "GDN_ERR_SHAPE") for n in ("q_stride", "q_head_stride", "k_stride", "k_head_stride",
                                                                   "v_stride", "v_head_stride")]]:
        assert append(lib, append_dims(**kw), cache()) == code, kw
    for name in APPEND:
        assert append(lib, append_dims(), cache(), **{name: FAKE + 1}) == "GDN_ERR_ALIGN", name
        if name not in ("q_weight", "k_weight"):
            assert append(lib, append_dims(), cache(), **{name: None}) == "GDN_ERR_NULL", name
    for kw in (dict(in_dtype=1), dict(q_stride=2048), dict(q_head_stride=256)):  # in place only where q is what q_out is
        assert append(lib, append_dims(**kw), cache(), q=FAKE, q_out=FAKE) == "GDN_ERR_SHAPE"
    assert status(lib.gdn_kv_append(None, cache(), *[FAKE] * 9, None)) == "GDN_ERR_NULL"
    assert append(lib, append_dims(), None) == "GDN_ERR_NULL"
    assert append(lib, append_dims(T=0), cache(), **dict.fromkeys(APPEND)) == "GDN_OK"


COMMIT = ["anc", "accepted", "table", "length", "new_length", "seq_status"]


def commit(lib, d, caches, n=None, **over):
    a = {name: FAKE + 256 * i for i, name in enumerate(COMMIT)}
    a.update(over)
    array = (attn.KvCacheStruct * len(caches))(*caches) if caches is not None else None
    return status(lib.gdn_kv_commit(d, array, len(caches or ()) if n is None else n, *(a[x] for x in COMMIT), None))


def test_commit_rejects(lib):
    def d(**kw):
        return attn.CommitDims(**{**dict(B=3, N=20, max_pages=40, reserved=0, table_stride=40), **kw})

    for kw, code in BAD_CACHE:
        assert commit(lib, d(), [cache(**kw)]) == code, kw
    for kw in (dict(B=-1), dict(B=65536), dict(N=-1), dict(N=257), dict(max_pages=-1), dict(max_pages=1 << 27), dict(reserved=1),
               dict(table_stride=-1)):
        assert commit(lib, d(**kw), [cache()]) == "GDN_ERR_SHAPE", kw
    for kw in (dict(n_pages=9), dict(page_size=8), dict(H_kv=1), dict(d=64), dict(dtype=2), dict(k_page_stride=8192),
               dict(v_row_stride=512), dict(v_head_stride=256)):
        assert commit(lib, d(), [cache(), cache(**kw)]) == "GDN_ERR_SHAPE", kw
    for name in COMMIT:
        assert commit(lib, d(), [cache()], **{name: FAKE + 2}) == "GDN_ERR_ALIGN"
        if name != "seq_status":
            assert commit(lib, d(), [cache()], **{name: None}) == "GDN_ERR_NULL"
    assert commit(lib, d(), [cache()], new_length=FAKE, length=FAKE) == "GDN_ERR_SHAPE"
    assert commit(lib, d(), [cache()], n=0) == "GDN_ERR_SHAPE"
    assert commit(lib, None, [cache()]) == "GDN_ERR_NULL"
    assert commit(lib, d(), None, n=1) == "GDN_ERR_NULL"
    assert commit(lib, d(B=0), [cache()], **dict.fromkeys(COMMIT)) == "GDN_OK"


def test_workspaces_have_room_for_every_part(lib):
    """two parts for each workgroup that the GPU has room for, fewer for small calls, none where a table has room for one unit"""
    assert need(lib, "decode", dims(max_pages=8), cache()) == need(lib, "verify", dims(max_pages=4), cache()) == 0
    assert need(lib, "decode", dims(max_pages=9), cache()) > 0
    for kind, d in (("decode", dims(B=1000, max_pages=1 << 20)), ("prefill", dims(T=10 ** 6)), ("verify", dims(B=60000))):
        rows = 16 if kind == "decode" else 128
        assert need(lib, kind, d, cache()) == 2 * 512 * rows * 130 * 4  # rows of 128 + 2
        assert 0 < need(lib, kind, dims(B=1, T=1, max_pages=16), cache()) < 2 * 64 * rows * 130 * 4
    # trees of 5 tiles: teams of 5; more tiles than fit at once: whole tiles only
    assert need(lib, "verify", dims(B=100, T=160), cache()) == 2 * (512 // 5) * 5 * 128 * 130 * 4
    assert need(lib, "verify", dims(T=256, H_q=2 * 300, q_stride=76800), cache()) == 0


def test_binding_has_no_cpu_fallback():
    src = open(attn.__file__).read()
    assert "oracle" not in src and "numpy" not in src


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not installed")
def test_attn_host_code_under_sanitizers(tmp_path):
    exe = str(tmp_path / "attn_driver")
    csrc = os.path.join(ROOT, "gated_deltanet_tree_gdn_amd", "csrc")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                        "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", csrc,
                        os.path.join(csrc, "gdn_attn_api.cpp"),
                        os.path.join(ROOT, "tests", "sanitize", "attn_driver.cpp"), "-o", exe],
                       capture_output=True, text=True)
    if r.returncode != 0 and "cannot find" in r.stderr and "asan" in r.stderr.lower():
        pytest.skip("sanitizer runtime not installed")
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60,
                       env=dict(os.environ, UBSAN_OPTIONS="print_stacktrace=1"))
    assert r.returncode == 0, r.stdout + r.stderr
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr
