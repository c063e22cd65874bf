// page_table.cpp -- the host page table of include/hb_cache.h: which pages
// each sequence holds, with reference counts, so that a fork shares pages, a
// write to a shared page copies it first, and compaction moves each page once
// however many sequences hold it.
#include <algorithm>
#include <map>
#include <new>
#include <set>
#include <vector>

#include "hb_cache.h"

namespace {

constexpr int kPage = 16;  // tokens a page

struct Seq {
    int n_tokens = 0;
    std::vector<int32_t> pages;
};

}  // namespace

struct hb_pages {
    std::vector<int> refs;   // sequences that hold each page
    std::set<int32_t> free;  // ordered: the lowest id is handed out first
    std::map<int, Seq> seqs;
};

extern "C" int hb_pages_create(int num_blocks, hb_pages **out)
{
    if (!out)
        return HB_EINVAL;
    *out = nullptr;
    if (num_blocks < 1)
        return HB_EINVAL;
    hb_pages *p = nullptr;
    try {
        p = new hb_pages();
        p->refs.assign((size_t)num_blocks, 0);
        for (int32_t b = 0; b < num_blocks; ++b)
            p->free.insert(p->free.end(), b);
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
        if (take > p->free.size())
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
            const int32_t b = *p->free.begin();
            p->free.erase(p->free.begin());
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
    // a page leaves the sequence before it becomes free, so a failed
    // allocation leaves every count as true as before
    std::vector<int32_t> &pages = it->second.pages;
    try {
        while (!pages.empty()) {
            const int32_t b = pages.back();
            if (p->refs[b] == 1)
                p->free.insert(b);
            --p->refs[b];
            pages.pop_back();
            it->second.n_tokens = std::min(it->second.n_tokens, (int)pages.size() * kPage);
        }
    } catch (...) {
        return HB_ENOMEM;
    }
    p->seqs.erase(it);
    return HB_OK;
}

extern "C" int hb_pages_compact(hb_pages *p, int32_t *src, int32_t *dst, int max_moves)
{
    if (!p || max_moves < 0 || (max_moves > 0 && (!src || !dst)))
        return HB_EINVAL;
    try {
        // what moves: the highest held pages to the lowest free ones.  All
        // destinations were free and all sources held, so none is both.
        std::vector<int32_t> where(p->refs.size(), -1);
        int n = 0;
        int32_t hi = (int32_t)p->refs.size() - 1;
        for (auto f = p->free.begin(); f != p->free.end() && n < max_moves; ++f) {
            while (hi > *f && p->refs[hi] == 0)
                --hi;
            if (hi <= *f)
                break;
            src[n] = hi;
            dst[n] = *f;
            where[hi] = *f;
            ++n;
            --hi;
        }
        // a page's node moves with it inside the set, without allocation
        for (int i = 0; i < n; ++i) {
            auto node = p->free.extract(dst[i]);
            node.value() = src[i];
            p->free.insert(std::move(node));
            p->refs[dst[i]] = p->refs[src[i]];
            p->refs[src[i]] = 0;
        }
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

extern "C" int hb_pages_num_free(hb_pages *p) { return p ? (int)p->free.size() : HB_EINVAL; }

extern "C" int hb_pages_refcount(hb_pages *p, int block)
{
    if (!p)
        return HB_EINVAL;
    if (block < 0 || (size_t)block >= p->refs.size())
        return HB_ERANGE;
    return p->refs[block];
}
