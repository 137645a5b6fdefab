// block_manager.cpp -- host-side block manager of a paged KV cache (declared in
// include/pagedkv.h, pa_bm_*): a pool of fixed-size physical blocks, one block table per
// sequence, reference counts, on-demand allocation, copy-on-write on divergence, and
// release back to the pool.
//
// Follows "PagedAttention in Production: Boosting LLM Serving Throughput with Paged KV
// Cache", section "Core Principle" (logical blocks map to physical blocks through a
// per-request block table; blocks are allocated on demand and returned to the pool when
// the request finishes); "Paged Attention and Memory Efficiency in Production LLM
// Serving", section "How PagedAttention borrows OS paging" (requests with an identical
// prefix point at the same physical blocks and a new block is allocated only when a
// sequence diverges, as in copy-on-write); "PagedAttention -- The KV Cache Problem",
// sections "How It Works" (fixed-size blocks, allocate on demand, free immediately) and
// "Why This Matters for Production" (parallel sampling and beam search share blocks
// copy-on-write).
//
// It produces what the CUDA calls consume: int32 block tables, int32 context lengths,
// int64 slot mappings and int32 (src, dst) copy pairs.  Not thread-safe: a caller
// serialises calls on one manager.
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <new>
#include <unordered_map>
#include <unordered_set>
#include <vector>

#include "pagedkv.h"

struct pa_block_manager {
  struct Seq {
    std::vector<int32_t> table;  // logical block i -> physical block
    int64_t len = 0;             // cached tokens
    bool swapped = false;        // preempted: holds no block, keeps its length
    int64_t holes = 0;           // table entries that are -1 (pages behind a window)
    std::vector<uint8_t> hole;   // while swapped: which entries were
  };
  int32_t num_blocks = 0, block_size = 0;
  std::vector<int32_t> ref;      // reference count per physical block
  // free blocks, handed out from the front: a ring with room for all of them, so that neither
  // taking nor giving back a block allocates
  std::vector<int32_t> ring;
  int32_t head = 0, num_free = 0;
  std::unordered_map<int32_t, Seq> seqs;
  int32_t next_id = 0;

  void push_free(int32_t b) {
    const int64_t at = (int64_t)head + num_free++;
    ring[(size_t)(at < num_blocks ? at : at - num_blocks)] = b;
  }
  int32_t take() {               // caller has checked that a block is free
    const int32_t b = ring[(size_t)head];
    head = head + 1 < num_blocks ? head + 1 : 0;
    --num_free;
    ref[(size_t)b] = 1;
    return b;
  }
  Seq* find(int32_t id) {
    auto it = seqs.find(id);
    return it == seqs.end() ? nullptr : &it->second;
  }
  const Seq* find(int32_t id) const {
    auto it = seqs.find(id);
    return it == seqs.end() ? nullptr : &it->second;
  }
  // a sequence that holds its blocks (known and not swapped out)
  const Seq* resident(int32_t id) const {
    const Seq* s = find(id);
    return s && !s->swapped ? s : nullptr;
  }
  void drop(int32_t b) {         // one reference less; a block nobody holds is free again
    if (--ref[(size_t)b] == 0) push_free(b);
  }
  int64_t blocks_for(int64_t tokens) const { return (tokens + block_size - 1) / block_size; }
};

namespace {

// No exception leaves a C entry.  The calls allocate all they need before their first change, so
// that one which runs out of memory has changed nothing.
template <typename Fn>
pa_status guarded(Fn fn) {
  try {
    return fn();
  } catch (...) {
    return PA_ERR_NO_MEMORY;
  }
}

}  // namespace

extern "C" {

pa_status pa_bm_create(int num_blocks, int block_size, const int32_t* free_order,
                       pa_block_manager** out) {
  if (!out) return PA_ERR_INVALID;
  *out = nullptr;
  if (num_blocks <= 0 || block_size <= 0) return PA_ERR_INVALID;
  pa_block_manager* bm = new (std::nothrow) pa_block_manager();
  if (!bm) return PA_ERR_NO_MEMORY;
  const pa_status r = guarded([&] {
    bm->num_blocks = num_blocks;
    bm->block_size = block_size;
    bm->ref.assign((size_t)num_blocks, 0);
    bm->ring.resize((size_t)num_blocks);
    if (!free_order) {
      for (int i = 0; i < num_blocks; ++i) bm->push_free(i);
      return PA_OK;
    }
    std::vector<uint8_t> seen((size_t)num_blocks, 0);
    for (int i = 0; i < num_blocks; ++i) {
      const int32_t b = free_order[i];
      if (b < 0 || b >= num_blocks || seen[(size_t)b]) return PA_ERR_INVALID;   // no permutation
      seen[(size_t)b] = 1;
      bm->push_free(b);
    }
    return PA_OK;
  });
  if (r != PA_OK) {
    delete bm;
    return r;
  }
  *out = bm;
  return PA_OK;
}

void pa_bm_destroy(pa_block_manager* bm) { delete bm; }

int pa_bm_free_blocks(const pa_block_manager* bm) { return bm ? bm->num_free : -1; }

int pa_bm_refcount(const pa_block_manager* bm, int block) {
  if (!bm || block < 0 || block >= bm->num_blocks) return -1;
  return bm->ref[(size_t)block];
}

pa_status pa_bm_allocate(pa_block_manager* bm, int num_tokens, int32_t* seq_id) {
  if (!bm || !seq_id || num_tokens < 0) return PA_ERR_INVALID;
  const int64_t need = bm->blocks_for(num_tokens);
  if (need > bm->num_free) return PA_ERR_NO_BLOCKS;
  return guarded([&] {
    pa_block_manager::Seq fresh;
    fresh.table.reserve((size_t)need);
    pa_block_manager::Seq& s = bm->seqs.emplace(bm->next_id, std::move(fresh)).first->second;
    for (int64_t i = 0; i < need; ++i) s.table.push_back(bm->take());
    s.len = num_tokens;
    *seq_id = bm->next_id++;
    return PA_OK;
  });
}

pa_status pa_bm_fork(pa_block_manager* bm, int32_t seq, int32_t* child) {
  if (!bm || !child) return PA_ERR_INVALID;
  const pa_block_manager::Seq* p = bm->resident(seq);
  if (!p) return PA_ERR_INVALID;
  return guarded([&] {
    // shares every block of the parent (whose place in the map does not move)
    const pa_block_manager::Seq& c = bm->seqs.emplace(bm->next_id, *p).first->second;
    for (int32_t b : c.table)
      if (b >= 0) ++bm->ref[(size_t)b];
    *child = bm->next_id++;
    return PA_OK;
  });
}

pa_status pa_bm_append_tokens(pa_block_manager* bm, const int32_t* seqs, int n, int64_t* slots,
                              int32_t* cow_pairs, int* num_cow) {
  if (!bm || n < 0 || (n && (!seqs || !slots || !cow_pairs || !num_cow))) return PA_ERR_INVALID;
  if (num_cow) *num_cow = 0;
  if (n == 0) return PA_OK;
  return guarded([&] {
    // Dry run on copies of the touched state: how many fresh blocks the whole batch needs
    // (a new logical block, or a private copy of a shared partial block), so that a batch
    // the pool cannot serve changes nothing.
    struct Sim {
      int64_t len, nblk;
      std::vector<int64_t> priv;   // logical blocks made private earlier in this batch
    };
    std::unordered_map<int32_t, Sim> sim;
    std::unordered_map<int32_t, int32_t> ref;
    int64_t need = 0;
    for (int i = 0; i < n; ++i) {
      const pa_block_manager::Seq* s = bm->resident(seqs[i]);
      if (!s) return PA_ERR_INVALID;
      Sim& m = sim.try_emplace(seqs[i], Sim{s->len, (int64_t)s->table.size(), {}}).first->second;
      const int64_t lb = m.len / bm->block_size;
      if (lb == m.nblk) {
        ++need;
        ++m.nblk;
        m.priv.push_back(lb);
      } else {
        bool priv = false;
        for (int64_t x : m.priv) priv |= x == lb;
        if (!priv) {
          const int32_t b = s->table[(size_t)lb];
          auto ri = ref.find(b);
          const int32_t r = ri == ref.end() ? bm->ref[(size_t)b] : ri->second;
          if (r > 1) {
            ++need;
            ref[b] = r - 1;
            m.priv.push_back(lb);
          }
        }
      }
      ++m.len;
    }
    if (need > bm->num_free) return PA_ERR_NO_BLOCKS;
    for (auto& [id, m] : sim) {              // room for the new entries, doubled as they grow
      std::vector<int32_t>& t = bm->find(id)->table;
      if (t.capacity() < (size_t)m.nblk) t.reserve(std::max((size_t)m.nblk, 2 * t.capacity()));
    }
    int nc = 0;
    for (int i = 0; i < n; ++i) {
      pa_block_manager::Seq& s = *bm->find(seqs[i]);
      const int64_t pos = s.len;
      const int64_t lb = pos / bm->block_size, off = pos % bm->block_size;
      if (lb == (int64_t)s.table.size()) {
        s.table.push_back(bm->take());
      } else if (bm->ref[(size_t)s.table[(size_t)lb]] > 1) {
        const int32_t src = s.table[(size_t)lb];
        const int32_t dst = bm->take();
        --bm->ref[(size_t)src];
        s.table[(size_t)lb] = dst;
        cow_pairs[2 * nc] = src;
        cow_pairs[2 * nc + 1] = dst;
        ++nc;
      }
      s.len = pos + 1;
      slots[i] = (int64_t)s.table[(size_t)lb] * bm->block_size + off;
    }
    *num_cow = nc;
    return PA_OK;
  });
}

pa_status pa_bm_release(pa_block_manager* bm, int32_t seq) {
  if (!bm) return PA_ERR_INVALID;
  auto it = bm->seqs.find(seq);
  if (it == bm->seqs.end()) return PA_ERR_INVALID;
  for (int32_t b : it->second.table)
    if (b >= 0) bm->drop(b);
  bm->seqs.erase(it);
  return PA_OK;
}

int64_t pa_bm_context_len(const pa_block_manager* bm, int32_t seq) {
  const pa_block_manager::Seq* s = bm ? bm->find(seq) : nullptr;
  return s ? s->len : -1;
}

int pa_bm_num_blocks_of(const pa_block_manager* bm, int32_t seq) {
  const pa_block_manager::Seq* s = bm ? bm->find(seq) : nullptr;
  return s ? (int)((int64_t)s->table.size() - (s->swapped ? 0 : s->holes)) : -1;
}

int pa_bm_max_blocks(const pa_block_manager* bm, const int32_t* seqs, int n) {
  if (!bm || n < 0 || (n && !seqs)) return -1;
  int mx = 0;
  for (int i = 0; i < n; ++i) {
    const pa_block_manager::Seq* s = bm->find(seqs[i]);
    if (!s) return -1;
    if ((int)s->table.size() > mx) mx = (int)s->table.size();
  }
  return mx;
}

pa_status pa_bm_block_tables(const pa_block_manager* bm, const int32_t* seqs, int n, int width,
                             int32_t fill, int32_t* tables, int32_t* context_lens) {
  if (!bm || n < 0 || width <= 0 || (n && (!seqs || !tables))) return PA_ERR_INVALID;
  for (int i = 0; i < n; ++i) {
    const pa_block_manager::Seq* s = bm->resident(seqs[i]);
    if (!s || (int64_t)s->table.size() > width || s->len > INT32_MAX) return PA_ERR_INVALID;
  }
  for (int i = 0; i < n; ++i) {
    const pa_block_manager::Seq* s = bm->find(seqs[i]);
    int32_t* row = tables + (int64_t)i * width;
    const size_t k = s->table.size();
    if (k) std::memcpy(row, s->table.data(), k * sizeof(int32_t));
    for (int j = (int)k; j < width; ++j) row[j] = fill;
    if (context_lens) context_lens[i] = (int32_t)s->len;
  }
  return PA_OK;
}

pa_status pa_bm_slot_of(const pa_block_manager* bm, int32_t seq, int64_t pos, int64_t* slot) {
  const pa_block_manager::Seq* s = bm ? bm->resident(seq) : nullptr;
  if (!s || !slot || pos < 0 || pos >= s->len) return PA_ERR_INVALID;
  const int32_t b = s->table[(size_t)(pos / bm->block_size)];
  if (b < 0) return PA_ERR_INVALID;                // its page was given back
  *slot = (int64_t)b * bm->block_size + pos % bm->block_size;
  return PA_OK;
}

// Preemption ("Paged Attention and Memory Efficiency in Production LLM Serving", section
// "Why KV cache memory was the bottleneck": in-flight requests are preempted when the
// cache runs out): the sequence's blocks go back to the pool as on release, after the
// caller has saved their contents; it keeps its id and length and later takes fresh
// blocks for the saved contents.
pa_status pa_bm_swap_out(pa_block_manager* bm, int32_t seq, int32_t* blocks, int* num_blocks) {
  if (!bm || !num_blocks) return PA_ERR_INVALID;
  pa_block_manager::Seq* s = bm->find(seq);
  if (!s || s->swapped || (!s->table.empty() && !blocks)) return PA_ERR_INVALID;
  if (s->holes) {
    const pa_status r = guarded([&] {
      s->hole.assign(s->table.size(), 0);
      return PA_OK;
    });
    if (r != PA_OK) return r;
  }
  size_t n = 0;
  for (size_t i = 0; i < s->table.size(); ++i) {
    if (s->table[i] >= 0) blocks[n++] = s->table[i];
    else s->hole[i] = 1;
  }
  for (int32_t b : s->table)
    if (b >= 0) bm->drop(b);
  s->table.clear();
  s->swapped = true;
  *num_blocks = (int)n;
  return PA_OK;
}

pa_status pa_bm_swap_in(pa_block_manager* bm, int32_t seq, int32_t* blocks, int* num_blocks) {
  if (!bm || !num_blocks) return PA_ERR_INVALID;
  pa_block_manager::Seq* s = bm->find(seq);
  if (!s || !s->swapped) return PA_ERR_INVALID;
  const int64_t all = bm->blocks_for(s->len), need = all - s->holes;
  if (need && !blocks) return PA_ERR_INVALID;
  if (need > bm->num_free) return PA_ERR_NO_BLOCKS;
  const pa_status r = guarded([&] {
    s->table.resize((size_t)all);
    return PA_OK;
  });
  if (r != PA_OK) return r;
  int64_t k = 0;
  for (int64_t i = 0; i < all; ++i)
    s->table[(size_t)i] = s->holes && s->hole[(size_t)i] ? -1 : (blocks[k++] = bm->take());
  s->hole.clear();
  s->swapped = false;
  *num_blocks = (int)need;
  return PA_OK;
}

// Bounded caches ("Core Principle": blocks go back to the pool as soon as nothing needs them):
// pages that lie wholly behind a sliding window and past the first tokens, and pages that a
// compaction of the kept tokens empties.
pa_status pa_bm_drop_window(pa_block_manager* bm, int32_t seq, int window, int num_sinks,
                            int* num_dropped) {
  if (!bm || !num_dropped || window < 1 || num_sinks < 0) return PA_ERR_INVALID;
  pa_block_manager::Seq* s = bm->find(seq);
  if (!s || s->swapped) return PA_ERR_INVALID;
  const int64_t bs = bm->block_size, behind = s->len - window;   // positions < behind are
  int n = 0;
  for (int64_t i = (num_sinks + bs - 1) / bs; (i + 1) * bs <= behind; ++i) {
    int32_t& b = s->table[(size_t)i];
    if (b < 0) continue;
    bm->drop(b);
    b = -1;
    ++s->holes;
    ++n;
  }
  *num_dropped = n;
  return PA_OK;
}

pa_status pa_bm_compact(pa_block_manager* bm, const int32_t* seqs, const int32_t* new_lens, int n,
                        int width, int32_t fill, int32_t* tables) {
  if (!bm || n < 0 || (n && (!seqs || !new_lens || !tables || width <= 0))) return PA_ERR_INVALID;
  return guarded([&] {
    // every sequence once, and what the batch needs: a new table keeps the entries that its
    // sequence alone holds (counts as they are before the call, so that a block that two
    // sequences of the batch share is a source for both and a destination for neither)
    std::unordered_set<int32_t> once;
    std::vector<std::vector<int32_t>> fresh((size_t)n);   // new tables, -1: a fresh block
    int64_t need = 0;
    for (int i = 0; i < n; ++i) {
      const pa_block_manager::Seq* s = bm->resident(seqs[i]);
      if (!s || new_lens[i] < 0 || new_lens[i] > s->len || !once.insert(seqs[i]).second)
        return PA_ERR_INVALID;
      const int64_t nb = bm->blocks_for(new_lens[i]);
      if (nb > width) return PA_ERR_INVALID;
      std::vector<int32_t>& t = fresh[(size_t)i];
      t.resize((size_t)nb);
      for (int64_t j = 0; j < nb; ++j) {
        const int32_t b = s->table[(size_t)j];
        const bool own = b >= 0 && bm->ref[(size_t)b] == 1;
        t[(size_t)j] = own ? b : -1;
        need += !own;
      }
    }
    if (need > bm->num_free) return PA_ERR_NO_BLOCKS;
    // fresh blocks first, from the front of the queue; what is left over goes to its back
    for (int i = 0; i < n; ++i)
      for (int32_t& b : fresh[(size_t)i])
        if (b < 0) b = bm->take();
    for (int i = 0; i < n; ++i) {
      pa_block_manager::Seq& s = *bm->find(seqs[i]);
      std::vector<int32_t>& t = fresh[(size_t)i];
      for (size_t j = 0; j < s.table.size(); ++j)
        if (s.table[j] >= 0 && (j >= t.size() || t[j] != s.table[j])) bm->drop(s.table[j]);
      int32_t* row = tables + (int64_t)i * width;
      for (int j = 0; j < width; ++j) row[j] = j < (int)t.size() ? t[(size_t)j] : fill;
      s.table.swap(t);
      s.len = new_lens[i];
      s.holes = 0;
    }
    return PA_OK;
  });
}

}  // extern "C"

// ---------------------------------------------------------------------------------------
// Cascade planning: which sequences of a batch read the same physical blocks at the start
// of their tables ("How PagedAttention borrows OS paging": requests with an identical
// prefix point their block tables at the same physical blocks), grouped into chunks whose
// members' query rows pa_decode_cascade decodes together over the shared prefix.
// ---------------------------------------------------------------------------------------
namespace {

constexpr int kCascadeMaxRows = 64;     // query rows a prefix chunk holds (group x members)

// Rows of one batch: table row i (entries row(i)[0..nblk(i))) and its length.
template <typename RowFn, typename LenFn>
pa_status plan_rows(int n, int block_size, int group, int chunk_width, RowFn row, LenFn len,
                    int32_t* prefix_lens, int32_t* chunk_members, int32_t* chunk_prefix_lens,
                    int* num_chunks, int* width_out) {
  if (n < 0 || block_size <= 0 || group <= 0 || !num_chunks ||
      (n && (!prefix_lens || !chunk_members || !chunk_prefix_lens)))
    return PA_ERR_INVALID;
  const int wmax = std::max(1, kCascadeMaxRows / group);
  if (chunk_width > 0 && (int64_t)group * chunk_width > kCascadeMaxRows) return PA_ERR_UNSUPPORTED;
  *num_chunks = 0;
  // sharing groups: rows with a non-empty context whose first physical block is the same,
  // in order of first appearance, members in batch order
  std::unordered_map<int32_t, int> by_first;
  std::vector<std::vector<int>> groups;
  for (int i = 0; i < n; ++i) {
    prefix_lens[i] = 0;
    if (len(i) <= 0) continue;
    const int32_t b0 = row(i)[0];
    auto it = by_first.find(b0);
    if (it == by_first.end()) {
      by_first.emplace(b0, (int)groups.size());
      groups.push_back({i});
    } else {
      groups[(size_t)it->second].push_back(i);
    }
  }
  // each sharing group's prefix: the leading table entries common to every member,
  // capped at the shortest member (0: the group shares nothing)
  std::vector<int64_t> plens(groups.size(), 0);
  int fit = 0;      // the default width: the widest group's members spread evenly over the
                    // fewest chunks of at most wmax members
  for (size_t gi = 0; gi < groups.size(); ++gi) {
    const std::vector<int>& mem = groups[gi];
    if (mem.size() < 2) continue;
    int64_t minlen = INT64_MAX;
    for (int i : mem) minlen = std::min<int64_t>(minlen, len(i));
    const int64_t nb = (minlen + block_size - 1) / block_size;
    int64_t common = 0;
    const int32_t* r0 = row(mem[0]);
    while (common < nb) {
      bool same = true;
      for (int i : mem) same = same && row(i)[common] == r0[common];
      if (!same) break;
      ++common;
    }
    plens[gi] = std::min<int64_t>(common * block_size, minlen);
    if (plens[gi] == 0) continue;
    const int m = (int)mem.size(), k = (m + wmax - 1) / wmax;
    fit = std::max(fit, (m + k - 1) / k);
  }
  const int width = chunk_width > 0 ? chunk_width : (fit > 0 ? fit : wmax);
  if (width_out) *width_out = width;
  int nc = 0;
  for (size_t gi = 0; gi < groups.size(); ++gi) {
    const std::vector<int>& mem = groups[gi];
    const int64_t plen = plens[gi];
    if (mem.size() < 2 || plen == 0) continue;
    for (size_t k = 0; k < mem.size(); k += (size_t)width) {
      int32_t* out = chunk_members + (int64_t)nc * width;
      for (int j = 0; j < width; ++j) {
        const size_t m = k + (size_t)j;
        out[j] = m < mem.size() ? mem[m] : -1;
        if (m < mem.size()) prefix_lens[mem[m]] = (int32_t)plen;
      }
      chunk_prefix_lens[nc] = (int32_t)plen;
      ++nc;
    }
  }
  *num_chunks = nc;
  return PA_OK;
}

}  // namespace

extern "C" {

pa_status pa_plan_cascade(const int32_t* block_tables, int max_blocks_per_seq,
                          const int32_t* context_lens, int num_seqs, int block_size, int group,
                          int chunk_width, int32_t* prefix_lens, int32_t* chunk_members,
                          int32_t* chunk_prefix_lens, int* num_chunks, int* chunk_width_out) {
  if (block_size <= 0 || (num_seqs > 0 && (!block_tables || !context_lens || max_blocks_per_seq <= 0)))
    return PA_ERR_INVALID;
  for (int i = 0; i < num_seqs; ++i) {     // every table must hold its sequence's blocks
    const int64_t c = context_lens[i];
    if (c < 0 || (c + block_size - 1) / block_size > max_blocks_per_seq) return PA_ERR_INVALID;
    const int32_t* row = block_tables + (int64_t)i * max_blocks_per_seq;
    for (int64_t j = 0; j < (c + block_size - 1) / block_size; ++j)
      if (row[j] < 0) return PA_ERR_INVALID;       // a page that was given back
  }
  return guarded([&] {
    return plan_rows(
        num_seqs, block_size, group, chunk_width,
        [&](int i) { return block_tables + (int64_t)i * max_blocks_per_seq; },
        [&](int i) { return (int64_t)context_lens[i]; }, prefix_lens, chunk_members,
        chunk_prefix_lens, num_chunks, chunk_width_out);
  });
}

pa_status pa_bm_plan_cascade(const pa_block_manager* bm, const int32_t* seqs, int n, int group,
                             int chunk_width, int32_t* prefix_lens, int32_t* chunk_members,
                             int32_t* chunk_prefix_lens, int* num_chunks, int* chunk_width_out) {
  if (!bm || n < 0 || (n && !seqs)) return PA_ERR_INVALID;
  return guarded([&] {
    std::vector<const pa_block_manager::Seq*> rows((size_t)n);
    for (int i = 0; i < n; ++i) {
      rows[(size_t)i] = bm->resident(seqs[i]);
      if (!rows[(size_t)i] || rows[(size_t)i]->holes) return PA_ERR_INVALID;
    }
    return plan_rows(
        n, bm->block_size, group, chunk_width,
        [&](int i) { return rows[(size_t)i]->table.data(); },
        [&](int i) { return rows[(size_t)i]->len; }, prefix_lens, chunk_members,
        chunk_prefix_lens, num_chunks, chunk_width_out);
  });
}

}  // extern "C"
