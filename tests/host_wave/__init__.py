"""The attention layer's kernels built for the host (calls.cpp), and calls of them on guarded arrays."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(os.path.dirname(HERE))
CSRC = os.path.join(ROOT, "nvfp4_w4a4_quantized_05_amd", "csrc")
SOURCES = ("nvfp4_attn.hip", "nvfp4_attn_few.hip", "nvfp4_attn_many.hip", "nvfp4_kv_cache.hip", "nvfp4_rope.hip")

# kernel<<<grid, block, 0, stream>>>(  ->  host_launch(kernel, grid, block,
_LAUNCH = re.compile(r"(\w+(?:<[^<>()\n]*>)?|(?<=  )\([^;\n]*\))<<<(.+?), (\w[\w.]*|\d+), 0, stream>>>\(")


def clang():
    """A clang++ that builds for this machine, or None: the vector types of the sources are clang's."""
    for c in ("/opt/rocm/llvm/bin/clang++", shutil.which("clang++")):
        if c and os.path.exists(c):
            return c
    return None


def build(out_dir):
    """Compile the kernels' sources for the host; returns the library."""
    for name in os.listdir(CSRC):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        if name in SOURCES:
            text, n = _LAUNCH.subn(r"host_launch(\1, \2, \3, ", text)
            assert n and "<<<" not in text, f"{name}: a launch that is written otherwise"
        with open(os.path.join(out_dir, name), "w") as f:
            f.write(re.sub(r'asm volatile\("" : "\+a".*', ";", text))  # a hint about registers
    lib = os.path.join(out_dir, "libhost.so")
    # -fwrapv: whole numbers that overflow do so as the GPU's would
    cmd = [clang(), "-x", "c++", "-std=c++17", "-O1", "-march=native", "-ffp-contract=off", "-fwrapv", "-shared", "-fPIC", "-w",
           "-I", HERE, "-I", os.path.join(ROOT, "include"), "-I", str(out_dir), os.path.join(HERE, "calls.cpp"), "-o", lib]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    lib = ctypes.CDLL(lib)
    vp, i32, i64, f32, u64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_uint64
    lib.host_alloc.argtypes, lib.host_alloc.restype = [u64, i32], vp
    lib.host_free.argtypes, lib.host_free.restype = [vp, u64], None
    lib.host_attn_workspace.argtypes, lib.host_attn_workspace.restype = [i64, i32, i32, i32, i32], u64
    lib.host_attn_plan.argtypes, lib.host_attn_plan.restype = [i64, i32, i32, i32, i32, vp], None
    lib.host_attn.argtypes = [vp] * 6 + [i32] * 5 + [vp, i64, i32, vp, vp, i32, i64, vp, i64, i32, f32, vp, vp, i64, vp]
    lib.host_attn.restype = u64
    lib.host_attn_pieces.argtypes, lib.host_attn_pieces.restype = [i32] * 4 + [vp, vp, i32, i64, i32, i32, vp, i32], i32
    lib.host_kv.argtypes = [i32] + [vp] * 6 + [i32] * 5 + [vp, i64, i32, vp, vp, i32, i64, vp, vp, i64, i32]
    lib.host_kv.restype = u64
    lib.host_rope.argtypes = [vp, i32, i64, i64, i64, i64, i32, i32, i32, i32, vp, vp, f32, vp, i32, vp, i32, vp, i32, vp, vp]
    lib.host_rope.restype = u64
    return lib


class Arrays:
    """Copies of arrays between unmapped pages, at their end or at their beginning, until the object is closed."""

    def __init__(self, lib, at_end):
        self.lib, self.at_end, self.made = lib, at_end, []

    def put(self, a, name):
        """Address of a copy of `a`, which is then that memory."""
        a = np.ascontiguousarray(a)
        p = self.lib.host_alloc(a.nbytes, int(self.at_end))
        view = np.ctypeslib.as_array((ctypes.c_uint8 * a.nbytes).from_address(p)).view(a.dtype).reshape(a.shape)
        view[...] = a
        self.made.append((p, a.nbytes, name))
        return p, view

    def __enter__(self):
        return self

    def __exit__(self, *_):
        for p, nbytes, _ in self.made:
            self.lib.host_free(p, nbytes)
        self.made = []

    def checked(self, at):
        """A call's answer: 0, or the address of an access out of bounds."""
        assert at == 0, f"an access out of bounds, next to {self.owner(at)}"

    def owner(self, address):
        """What array an address lies next to."""
        return min(self.made, key=lambda m: max(m[0] - address, address - m[0] - m[1]))[2]


def bf16(x):
    """fp32 values as bf16 bits, round to nearest even (finite values)."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    return ((b + 0x7FFF + (b >> 16 & 1)) >> 16).astype(np.uint16)


def f32(b):
    """bf16 bits as fp32."""
    return (b.astype(np.uint32) << 16).view(np.float32)


def plan(lib, T, n_seqs, hk, group, d):
    out = (ctypes.c_int32 * 3)()
    lib.host_attn_plan(T, n_seqs, hk, group, d, out)
    return tuple(out)


def pieces(lib, rows, kv, hq, hk, d, page, max_pages, tree):
    """[n, 8]: range, sequence, tile, minor, first step, step behind the last, slot and the unit's steps of all work."""
    lens, cu = np.array(kv, dtype=np.int32), np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    out = np.zeros((1 << 16, 8), dtype=np.int64)
    n = lib.host_attn_pieces(page.bit_length() - 1, hk, d, max_pages, lens.ctypes.data, cu.ctypes.data, len(rows), int(cu[-1]), hq,
                             int(tree), out.ctypes.data, len(out))
    assert n <= len(out)
    return out[:n]


def _cache(mem, paged):
    """The arguments for a Paged cache and, by name, its arrays as the call will leave them."""
    fp4, args, left = paged.fmt == "nvfp4", [], {}
    for a, turned in (("codes", False), ("codes", True), ("scales", False), ("scales", True)):
        name = "kv"[turned]
        x = getattr(paged, a)[name]
        p, left[name, a] = mem.put(np.swapaxes(x, 2, 3) if turned else x, f"{name} {a}") if a == "codes" or fp4 else (None, x)
        args.append(p)
    args += [mem.put(np.array([paged.gs[n]], dtype=np.float32), n + "_gs")[0] for n in "kv"]
    args += [int(fp4), paged.n_pages, paged.page.bit_length() - 1, paged.hk, paged.d]
    table = mem.put(paged.table[:, :paged.max_pages], "page_table")[0]
    return args + [table, paged.max_pages, paged.max_pages], left


def _sequences(mem, rows, kv, cu, lead):
    lens = mem.put(np.array(kv, dtype=np.int32), "kv_lens")[0]
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32) + np.int32(lead)
    return [lens, mem.put(starts, "cu_seqlens")[0] if cu else None, len(rows)], starts


def kv_rows(lib, paged, rows, kv, k, v, *, write, cu=True, lead=0, at_end=True):
    """kv_cache_write of rows k and v [T, hk * d] (fp32, or bf16 bits), or _read in place of them.  Returns (k, v, the cache's
    arrays by (name, "codes" or "scales"), row-major)."""
    with Arrays(lib, at_end) as mem:
        cache, left = _cache(mem, paged)
        seqs, _ = _sequences(mem, rows, kv, cu, lead)
        (kp, k), (vp, v) = mem.put(k, "k rows"), mem.put(v, "v rows")
        mem.checked(lib.host_kv(int(write), *cache, *seqs, k.shape[0], kp, vp, k.shape[1], int(k.dtype == np.uint16)))
        return k.copy(), v.copy(), {n: (np.swapaxes(x, 2, 3) if n[0] == "v" and x.size else x).copy() for n, x in left.items()}


def attn(lib, paged, rows, kv, hq, q, *, tree=None, scale=None, cu=True, lead=0, tail=0, at_end=True):
    """The call on a tests.attn_util.Paged cache and bf16 bits q [T, hq * d].  Returns o as fp32; rows outside the sequences 7.5."""
    d, hk, T = paged.d, paged.hk, lead + sum(rows) + tail
    with Arrays(lib, at_end) as mem:
        cache, _ = _cache(mem, paged)
        seqs, starts = _sequences(mem, rows, kv, cu, lead)
        masks = None if tree is None else mem.put(np.concatenate([np.zeros(lead, np.int64), *tree, np.zeros(tail, np.int64)]), "tree")[0]
        o, out = mem.put(np.full((T, hq * d), 0x40F0, dtype=np.uint16), "o")
        need = lib.host_attn_workspace(T, len(rows), hq, hk, d)
        ws = mem.put(np.full(need // 4, np.nan, dtype=np.float32), "workspace")[0]
        mem.checked(lib.host_attn(*cache, *seqs, T, mem.put(q, "q")[0], hq * d, hq, d ** -0.5 if scale is None else scale, masks, o,
                                  hq * d, ws))
        return f32(out), starts


def rope(lib, x, q_w, k_w, table, pos, *, q_col, k_col, hq, hk, eps, pair_axis=None, adjacent=False, at_end=True):
    """The call on x (fp32, or bf16 bits) [T, cols]; pos [axes, T].  Returns q and k as fp32."""
    d, T = len(q_w), x.shape[0]
    axis = np.zeros(8, dtype=np.uint32)
    for p, n in enumerate(pair_axis or ()):
        axis[p // 16] |= np.uint32(n << p % 16 * 2)
    with Arrays(lib, at_end) as mem:
        q, qv = mem.put(np.zeros((T, hq * d), np.uint16), "q")
        k, kv = mem.put(np.zeros((T, hk * d), np.uint16), "k")
        mem.checked(lib.host_rope(mem.put(x, "x")[0], int(x.dtype == np.uint16), x.shape[1], q_col, k_col, T, hq, hk, d, table.shape[1],
                                  mem.put(q_w, "q_w")[0], mem.put(k_w, "k_w")[0], eps, mem.put(table, "cos_sin")[0], table.shape[0],
                                  mem.put(pos.astype(np.int32), "positions")[0], pos.shape[0], mem.put(axis, "axes")[0],
                                  int(adjacent), q, k))
        return f32(qv), f32(kv)
