"""csrc/sample.cuh on the CPU: its source, compiled by g++ on tests/cta_emulator.h
with the inline PTX replaced, run cluster by cluster under schedules that let one
warp or CTA run ahead of the others."""
from __future__ import annotations

import ctypes
import hashlib
import os
import re
import shutil
import subprocess

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = os.path.join(os.path.dirname(HERE), "q8_block_quantized_02_b200", "csrc", "sample.cuh")
THREADS, WARPS = 512, 16

# every asm statement of the source, by its instruction
PTX = [
    (r'asm volatile\("mov\.u32 %0, %%cluster_nctarank;" : "=r"\(([^)]*)\)\);', r"\1 = (uint32_t)emu::g->ctas;"),
    (r'asm volatile\("barrier\.cluster\.arrive\.\w+\.aligned;" ::: "memory"\);', "emu::cluster_arrive();"),
    (r'asm volatile\("barrier\.cluster\.wait\.\w+\.aligned;" ::: "memory"\);', "emu::cluster_wait();"),
    (r'asm volatile\("ld\.shared::cluster\.u(\d\d)[^;]*;" : "=[lr]"\(v\) : "r"\(addr\) : "memory"\);',
     r"v = *static_cast<uint\1_t *>(emu::at(addr, \1 / 8));"),
    (r'asm volatile\("st\.shared::cluster\.u(\d\d)[^;]*;" :: ?"r"\(addr\), "[lr]"\(v\) : "memory"\);',
     r"*static_cast<uint\1_t *>(emu::at(addr, \1 / 8)) = v;"),
    (r'asm volatile\("atom\.relaxed\.cluster\.shared::cluster\.add\.u32[^;]*;" : "=r"\(o\) : "r"\(addr\), "r"\(v\) : "memory"\);',
     "o = atomicAdd(static_cast<uint32_t *>(emu::at(addr, 4)), v);"),
]

DRIVER = r"""
static void body(const void *a) { q8::sample_kernel<1>(*static_cast<const q8::SampleArgs *>(a)); }
extern "C" const char *run_sample(const float *logits, const float *temperature, const int32_t *top_k, const float *top_p,
                                  const float *min_p, const float *u, int32_t *token, float *prob, int N, int V, int ld,
                                  int cl, const int *order, uint32_t rng, int fill) {
    static emu::Cluster c;
    q8::SampleArgs a{};
    a.logits = logits, a.temperature = temperature, a.top_k = top_k, a.top_p = top_p, a.min_p = min_p, a.u = u;
    a.token = token, a.prob = prob, a.ld = ld, a.V = V;
    a.slice = ((V + cl - 1) / cl + 3) / 4 * 4;
    for (int row = 0; row < N; ++row) {
        const char *e = emu::run(c, row, cl, q8::kSampleThreads, q8::sample_smem_bytes(a.slice, cl), order, rng, fill, body, &a);
        if (e[0]) return e;
    }
    return "";
}
"""


def host_source() -> str:
    """sample.cuh as C++ for the host."""
    text = open(SOURCE).read()
    text = re.sub(r"^#(include|pragma) .*$", "", text, flags=re.M)
    text = re.sub(r"extern __shared__ [^;]*\bsample_smem\[\];", "uint8_t *sample_smem = emu::smem();", text)
    for pattern, to in PTX:
        text = re.sub(pattern, to, text)
    left = [line for line in text.splitlines() if re.search(r"\basm\b", line)]
    assert not left, f"no host form for: {left}"
    return '#include "cta_emulator.h"\n' + text + DRIVER


def build(folder: str) -> ctypes.CDLL:
    """Compiles the emulated sampler into `folder`."""
    text = host_source()
    name = os.path.join(folder, "sample_" + hashlib.sha1(text.encode()).hexdigest()[:12])
    with open(name + ".cpp", "w") as f:
        f.write(text)
    # -ffp-contract=off: fused multiply-adds only where the source has them
    subprocess.run([shutil.which("g++"), "-std=c++17", "-O1", "-g", "-fPIC", "-shared", "-ffp-contract=off", "-fwrapv",
                    "-fno-strict-aliasing", "-fno-stack-protector", "-w", "-I", HERE, "-o", name + ".so", name + ".cpp"],
                   check=True)
    lib = ctypes.CDLL(name + ".so")
    lib.run_sample.restype = ctypes.c_char_p
    return lib


def orders(cl: int) -> dict:
    """Schedules: which warp runs ahead (cta * 16 + warp, the foremost first), and a seed for a random one."""
    n = cl * WARPS
    up = list(range(n))
    by_warp = [c * WARPS + w for w in range(WARPS) for c in range(cl)]
    return {"first warps ahead": (up, 0), "last warps ahead": (up[::-1], 0), "first warps of all CTAs ahead": (by_warp, 0),
            "last warps of all CTAs ahead": (by_warp[::-1], 0), "random": (up, 12345)}


def sample(lib, l, temperature=None, top_k=None, top_p=None, min_p=None, u=0.0, cl=1, order=None, V=None, fill=0xa5):
    """(token, prob) as q8_sample gives them; raises what the emulator finds."""
    l = np.ascontiguousarray(np.atleast_2d(l), np.float32)
    N, ld = l.shape
    V = ld if V is None else V

    def row(v, dt):
        return None if v is None else np.ascontiguousarray(np.broadcast_to(np.asarray(v, dt), (N,)))

    given = [row(temperature, np.float32), row(top_k, np.int32), row(top_p, np.float32), row(min_p, np.float32),
             row(u, np.float32)]
    token, prob = np.full(N, -99, np.int32), np.full(N, np.nan, np.float32)
    first, rng = order if order is not None else orders(cl)["first warps ahead"]
    ptr = lambda a: None if a is None else ctypes.c_void_p(a.ctypes.data)
    e = lib.run_sample(ptr(l), *[ptr(a) for a in given], ptr(token), ptr(prob), N, V, ld, cl,
                       (ctypes.c_int * len(first))(*first), ctypes.c_uint32(rng), fill)
    if e:
        raise RuntimeError(e.decode())
    return token, prob
