// Host-side planning of the cache calls (no device code): how a pool's pages are
// moved.  Kept apart from the kernels so that it can be built on its own, for
// instance with the host sanitizers.
#include "attention.h"

namespace cfp32 {

PageShape page_shape(const Pool &p)
{
    PageShape g;
    const int64_t eb = p.elem_bytes, page = (int64_t)1 << p.page_log2;
    auto rows = [&](const PagesView &v) { return PageRows{(char *)v.data, v.page * eb, v.head * eb, v.tok * eb}; };
    g.k = rows(p.k), g.v = rows(p.v);
    int64_t bytes = p.D * eb;
    auto whole = [&](const PagesView &v) {  // every value of a page in one run
        return (v.tok == p.D && (v.head == page * p.D || p.Hkv == 1)) || (v.head == p.D && (v.tok == p.Hkv * (int64_t)p.D || page == 1));
    };
    if (whole(p.k) && whole(p.v)) {
        bytes *= p.Hkv * page;
        g.n2 = 1, g.rows = 1;
    } else {
        g.n2 = (int)page;
        g.rows = p.Hkv * page;
    }
    int64_t a = bytes | 16 | (int64_t)(uintptr_t)g.k.data | (int64_t)(uintptr_t)g.v.data | g.k.page | g.v.page;
    if (g.rows > 1) a |= g.k.s1 | g.k.s2 | g.v.s1 | g.v.s2;
    g.vec_bytes = (int)(a & -a);
    g.vecs = bytes / g.vec_bytes;
    return g;
}

}  // namespace cfp32
