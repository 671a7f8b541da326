"""The pool's kept tensor maps where memory runs out: nothing is kept, and no exception leaves the call."""
import subprocess

from paged_kv_cache_223_gb300 import _build

ALLOCATE = r"""
#include <cstdlib>
#include <new>
bool none = false;
void *operator new(std::size_t n) {
    if (none) throw std::bad_alloc();
    return std::malloc(n);
}
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, std::size_t) noexcept { std::free(p); }
"""

MAPS = r"""
#include "pa_pool.h"
extern bool none;
int main() {
    std::unordered_map<const void *, CUtensorMap> maps;
    CUtensorMap m = {};
    static char at[9000];
    none = true;
    pa::keep_map(maps, at, m);
    none = false;
    if (!maps.empty()) return 1;
    for (char &c : at) {
        pa::keep_map(maps, &c, m);
        if (!maps.count(&c) || maps.size() > 4097) return 2;
    }
    return 0;
}
"""


def test_no_memory_for_a_map(tmp_path):
    sources = {tmp_path / "allocate.cpp": ALLOCATE, tmp_path / "maps.cu": MAPS}
    for path, text in sources.items():
        path.write_text(text)
    program = str(tmp_path / "maps")
    made = subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", f"-I{_build.INCLUDE}", f"-I{_build.PKG}/csrc", "-o", program,
                           *map(str, sources)], capture_output=True, text=True)
    assert made.returncode == 0, made.stderr
    assert subprocess.run([program], timeout=60).returncode == 0
