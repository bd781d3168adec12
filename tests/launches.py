"""What the library's entry points launch, on the host: a process in which a stand-in takes the HIP runtime's place writes
down each launch's kernel and grid, and runs nothing. Pointers given to the entry points are not read."""
import json
import os
import re
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Loaded before the library, with its names for all: the library's calls come here. Memory is an address that nothing reads.
STAND_IN = r"""
#include <stddef.h>
typedef struct { unsigned x, y, z; } dim3;
static struct { const void *f; const char *name; } known[4096];
static int count;
static dim3 grid, block;
static size_t shared;
static void *stream;
static struct { const char *name; unsigned v[4]; } launch[64];
static int launches;
int capturing, no_memory;
void clear(void) { launches = 0; }
int launched(void) { return launches; }
const char *name_of(int i) { return launch[i].name; }
unsigned size_of(int i, int k) { return launch[i].v[k]; }
void **__hipRegisterFatBinary(const void *p) { static void *module; (void)p; return &module; }
void __hipUnregisterFatBinary(void **m) { (void)m; }
void __hipRegisterVar(void **m, void *v, char *h, char *d, int e, size_t s, int c, int g) { (void)m, (void)v, (void)h, (void)d, (void)e, (void)s, (void)c, (void)g; }
void __hipRegisterFunction(void **m, const void *f, char *d, const char *name, unsigned t, void *a, void *b, void *c, void *e, int *w) {
    (void)m, (void)d, (void)t, (void)a, (void)b, (void)c, (void)e, (void)w;
    if (count < 4096) known[count].f = f, known[count++].name = name;
}
int __hipPushCallConfiguration(dim3 g, dim3 b, size_t s, void *t) { grid = g, block = b, shared = s, stream = t; return 0; }
int __hipPopCallConfiguration(dim3 *g, dim3 *b, size_t *s, void **t) { *g = grid, *b = block, *s = shared, *t = stream; return 0; }
int hipLaunchKernel(const void *f, dim3 g, dim3 b, void **args, size_t s, void *t) {
    (void)args, (void)s, (void)t;
    if (launches == 64) return 1;
    launch[launches].name = "";
    for (int i = 0; i < count; ++i)
        if (known[i].f == f) launch[launches].name = known[i].name;
    unsigned v[4] = {g.x, g.y, g.z, b.x};
    for (int k = 0; k < 4; ++k) launch[launches].v[k] = v[k];
    ++launches;
    return 0;
}
int hipDeviceGetAttribute(int *v, int a, int d) { (void)a, (void)d; *v = 256; return 0; }
int hipMalloc(void **p, size_t n) { (void)n; *p = (void *)0x100000; return no_memory; }
int hipFree(void *p) { (void)p; return 0; }
int hipGetDevice(int *d) { *d = 0; return 0; }
int hipSetDevice(int d) { (void)d; return 0; }
int hipGetLastError(void) { return 0; }
int hipGetSymbolAddress(void **p, const void *s) { (void)s; *p = (void *)0x100000; return 0; }
int hipStreamGetDevice(void *t, int *d) { (void)t; *d = 0; return 0; }
int hipStreamIsCapturing(void *t, int *c) { (void)t; *c = capturing; return 0; }
int hipStreamSynchronize(void *t) { (void)t; return 0; }
"""

CHILD = """
import ctypes, json, sys
here = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
here.name_of.restype = ctypes.c_char_p
sys.modules["torch"] = type(sys)("torch")   # not the real one: its kernels are many, and all would register
import fp32_gemm_nn_amd as mg
mg.load_library()
out = []
for name, args, state in json.load(sys.stdin):
    for k in ("capturing", "no_memory"):
        ctypes.c_int.in_dll(here, k).value = state.get(k, 0)
    here.clear()
    rc = getattr(mg, name)(*args)
    out.append([rc, [[here.name_of(i).decode(), *(here.size_of(i, k) for k in range(4))] for i in range(here.launched())]])
json.dump(out, sys.stdout)
"""


class Launch:
    """A kernel by its name and the numbers of its template (truth values and enumerators too), its grid, and its threads."""

    def __init__(self, name, x, y, z, threads):
        self.name, self.grid, self.threads = name, (x, y, z), threads
        template = re.search(r"\d([a-z][a-z0-9_]*)I", name)
        self.kernel = template.group(1) if template else name
        self.numbers = [int(v) for v in re.findall(r"L(?:i|b|N\w*?E)(\d+)E", name)]

    def __repr__(self):
        return f"{self.kernel}{self.numbers} {self.grid}"


def launches(calls, folder):
    """For each (C name, arguments, state) the status and its launches, of one process. state: {"capturing": 1} or {"no_memory": 1}, or {}."""
    lib = os.path.join(str(folder), "stand_in.so")
    source = os.path.join(str(folder), "stand_in.c")
    with open(source, "w") as f:
        f.write(STAND_IN)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", source, "-o", lib], check=True)
    done = subprocess.run([sys.executable, "-c", CHILD, lib], input=json.dumps(calls), cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
    return [(rc, [Launch(*v) for v in got]) for rc, got in json.loads(done.stdout)]
