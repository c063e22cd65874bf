// page_table.cpp -- the host page table of include/hb_cache.h: which pages
// each sequence holds, with reference counts, so that a fork shares pages, a
// write to a shared page copies it first, and compaction moves each page once
// however many sequences hold it.
#include <stdint.h>

#include <algorithm>
#include <map>
#include <new>
#include <vector>

#include "hb_cache.h"

namespace {

constexpr int kPage = 16;                   // tokens a page
constexpr int kMaxPages = (1 << 27) - 1;    // slots (16 x page + offset) fit 32 bits

struct Seq {
    int n_tokens = 0;
    std::vector<int32_t> pages;
};

}  // namespace

struct hb_pages {
    std::vector<int> refs;       // sequences that hold each page
    std::vector<uint64_t> free;  // a bit for each page that none holds
    size_t first = 0;            // no word before it has a bit set
    int n_free = 0;
    std::map<int, Seq> seqs;

    void give(int32_t b)
    {
        free[b / 64] |= 1ull << (b % 64);
        first = std::min(first, (size_t)b / 64);
        ++n_free;
    }
    // The lowest free page; there is one.
    int32_t take()
    {
        while (!free[first])
            ++first;
        const int bit = __builtin_ctzll(free[first]);
        free[first] &= free[first] - 1;
        --n_free;
        return (int32_t)(first * 64 + bit);
    }
};

extern "C" int hb_pages_create(int num_blocks, hb_pages **out)
{
    if (!out)
        return HB_EINVAL;
    *out = nullptr;
    if (num_blocks < 1 || num_blocks > kMaxPages)
        return HB_EINVAL;
    hb_pages *p = nullptr;
    try {
        p = new hb_pages();
        p->refs.assign((size_t)num_blocks, 0);
        p->free.assign(((size_t)num_blocks + 63) / 64, ~0ull);
        if (num_blocks % 64)
            p->free.back() = (1ull << (num_blocks % 64)) - 1;
        p->n_free = num_blocks;
    } catch (...) {
        delete p;
        return HB_ENOMEM;
    }
    *out = p;
    return HB_OK;
}

extern "C" void hb_pages_destroy(hb_pages *p) { delete p; }

extern "C" int hb_pages_extend(hb_pages *p, int seq, int n_tokens, int32_t *copy_src, int32_t *copy_dst)
{
    if (!p || !copy_src || !copy_dst || n_tokens < 0)
        return HB_EINVAL;
    *copy_src = *copy_dst = -1;
    try {
        auto it = p->seqs.find(seq);
        const bool fresh = it == p->seqs.end();
        const int have = fresh ? 0 : it->second.n_tokens;
        if (n_tokens < have)
            return HB_EINVAL;
        const size_t held = fresh ? 0 : it->second.pages.size();
        const size_t want = ((size_t)n_tokens + kPage - 1) / kPage;
        // the first new token's page, if it is part-filled and shared
        const bool copy = n_tokens > have && have % kPage != 0 && p->refs[it->second.pages[held - 1]] > 1;
        const size_t take = want - held + (copy ? 1 : 0);
        if (take > (size_t)p->n_free)
            return HB_ENOMEM;
        // everything that may throw comes before the first change
        if (fresh)
            it = p->seqs.emplace(seq, Seq()).first;
        Seq &s = it->second;
        try {
            s.pages.reserve(want);
        } catch (...) {
            if (fresh)
                p->seqs.erase(it);
            throw;
        }
        auto next = [&]() {
            const int32_t b = p->take();
            p->refs[b] = 1;
            return b;
        };
        if (copy) {
            *copy_src = s.pages[held - 1];
            --p->refs[*copy_src];
            s.pages[held - 1] = *copy_dst = next();
        }
        while (s.pages.size() < want)
            s.pages.push_back(next());
        s.n_tokens = n_tokens;
    } catch (...) {
        return HB_ENOMEM;
    }
    return HB_OK;
}

extern "C" int hb_pages_fork(hb_pages *p, int parent, int child, int n_tokens)
{
    if (!p)
        return HB_EINVAL;
    auto it = p->seqs.find(parent);
    if (it == p->seqs.end() || p->seqs.count(child) || n_tokens < -1 || n_tokens > it->second.n_tokens)
        return HB_EINVAL;
    try {
        Seq s;
        s.n_tokens = n_tokens < 0 ? it->second.n_tokens : n_tokens;
        const size_t n = ((size_t)s.n_tokens + kPage - 1) / kPage;
        s.pages.assign(it->second.pages.begin(), it->second.pages.begin() + n);
        Seq &c = p->seqs.emplace(child, Seq()).first->second;
        std::swap(c, s);
        for (int32_t b : c.pages)
            ++p->refs[b];
    } catch (...) {
        return HB_ENOMEM;
    }
    return HB_OK;
}

extern "C" int hb_pages_release(hb_pages *p, int seq)
{
    if (!p)
        return HB_EINVAL;
    auto it = p->seqs.find(seq);
    if (it == p->seqs.end())
        return HB_EINVAL;
    for (int32_t b : it->second.pages)
        if (--p->refs[b] == 0)
            p->give(b);
    p->seqs.erase(it);
    return HB_OK;
}

extern "C" int hb_pages_compact(hb_pages *p, int32_t *src, int32_t *dst, int max_moves)
{
    if (!p || max_moves < 0 || (max_moves > 0 && (!src || !dst)))
        return HB_EINVAL;
    try {
        // The highest held pages move to the lowest free ones.  All
        // destinations were free and all sources held, so none is both.
        std::vector<int32_t> where(p->refs.size(), -1);
        int n = 0;
        int32_t hi = (int32_t)p->refs.size() - 1;
        while (n < max_moves && p->n_free > 0) {
            while (p->first < p->free.size() && !p->free[p->first])
                ++p->first;
            const int32_t lo = (int32_t)(p->first * 64 + __builtin_ctzll(p->free[p->first]));
            while (hi > lo && p->refs[hi] == 0)
                --hi;
            if (hi <= lo)
                break;
            p->take();  // lo; what was held above it is given back below
            p->refs[lo] = p->refs[hi];
            p->refs[hi] = 0;
            src[n] = hi;
            dst[n] = lo;
            where[hi] = lo;
            ++n;
            --hi;
        }
        for (int i = 0; i < n; ++i)
            p->give(src[i]);
        for (auto &kv : p->seqs)
            for (int32_t &b : kv.second.pages)
                if (where[b] >= 0)
                    b = where[b];
        return n;
    } catch (...) {
        return HB_ENOMEM;
    }
}

extern "C" int hb_pages_table(hb_pages *p, int seq, int32_t *table, int max_blocks, int *n_tokens)
{
    if (!p || max_blocks < 0 || (max_blocks > 0 && !table))
        return HB_EINVAL;
    auto it = p->seqs.find(seq);
    if (it == p->seqs.end())
        return HB_EINVAL;
    const std::vector<int32_t> &pages = it->second.pages;
    std::copy(pages.begin(), pages.begin() + std::min(pages.size(), (size_t)max_blocks), table);
    if (n_tokens)
        *n_tokens = it->second.n_tokens;
    return (int)pages.size();
}

extern "C" int hb_pages_num_free(hb_pages *p) { return p ? p->n_free : HB_EINVAL; }

extern "C" int hb_pages_refcount(hb_pages *p, int block)
{
    if (!p)
        return HB_EINVAL;
    if (block < 0 || (size_t)block >= p->refs.size())
        return HB_ERANGE;
    return p->refs[block];
}
