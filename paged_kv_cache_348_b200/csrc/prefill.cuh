// prefill.cuh -- attention of ragged prompt chunks over a paged cache, with a sliding window
// and a few first tokens that stay visible, on the tcgen05 tensor cores.
//
// The operation is the one of decode.cuh ("Paged Attention and Memory Efficiency in
// Production LLM Serving", section "How PagedAttention borrows OS paging": the kernel
// resolves the block table, the arithmetic is the plain softmax(scale q K^T) V) for
// sequences with many new tokens: token i of n at position p = ctx - n + i sees the cached
// positions t <= p with t > p - window or t < num_sinks.
//
// What bounds it: with n new tokens every K/V row is used by up to n * group query rows, so
// past a few hundred rows it is the contractions (4 D flop per query row and visible
// position) and, next to them, one exponential per score: a 128 x 128 tile of scores costs
// the tensor cores 2 x 512 cycles at D = 128 and the special-function units (16 a cycle and
// SM) 1024, so the two have to run side by side.
//
//  * An item is the query rows of up to 2 floor(128 / group) new tokens of one (sequence, kv
//    head), as two subtiles of up to 128 rows (token-major: row = token * group + head of the
//    group, so the heads of a kv head share every K/V byte).  While the softmax of one subtile
//    runs, the tensor cores work on the other.
//  * Key tiles are 128 positions.  As in decode.cuh the first tokens are laid directly in
//    front of the window ("virtual" positions, rounded to 32), so a tile of a few first
//    tokens is not paid for on its own; positions between are neither loaded nor computed.
//  * Tensor memory, 512 columns: one S (128 columns) that the two subtiles use in turn, P of
//    either (64 columns, 16 bits a value, the A operand of P V from there) and O of either
//    (128).  A subtile's scores are taken to registers at once, so the next Q K^T need not
//    wait for its exponentials, and the tensor cores always have a product to run.
//  * Softmax: one thread per query row, base 2 in 32 bits, so a row's maximum and sum need
//    no exchange.  The reference maximum moves only when a score passes it by 2^8 (O is
//    then rescaled in tensor memory); after a row's first key tile that is rare.  The row
//    sum takes the weights before they are rounded to 16 bits.  A weight rounded to the
//    cache's type (bf16: half a step 2^-9..2^-8) is off by as much as the output's own
//    rounding; carrying its residual too, as decode does, would make P V half as fast in a
//    kernel that the tensor cores bound.
//  * Warps 0-3 and 4-7: softmax and output of the two subtiles; 8: one thread issues the
//    tensor-core operations; 9: K and V tiles by TMA through the block table into a ring of
//    tiles; 10: query rows; 11: hands out items.  Items go to CTAs as they become free (one
//    CTA an SM), since a causal prompt's items differ in length.
//  * Rows of V that no query of the sequence sees may hold anything (NaN times a weight of 0
//    would reach O): units that hold such rows are copied row by row with zeros in their
//    place, everything else comes by TMA boxes.  Scores are masked by selection.
//  * Every wait is bounded; tensor memory is released on every path.
#pragma once
#include <climits>

#include "decode_wide.cuh"

namespace pkv {

constexpr int DEV_BAD_QUERY = 0x40;
constexpr int kPfSub = 128;                       // query rows of a subtile (MMA M)
// new tokens of a subtile: whole tokens, so at most group - 1 of its rows are idle
__host__ __device__ constexpr int pf_tokens(int group) { return kPfSub / group; }
constexpr int kPfKeys = 128;                      // positions of a key tile
constexpr int kPfThreads = 384;
// of 16 pairs of weights, those not on ex2 (none against two: 24 ragged chunks 48.7 against 47.2
// us, two prompts of 4000 tokens 218 against 214.5, one of 8000 759 against 755; more were slower)
constexpr int kPfPoly = 2;
constexpr int kPfItems = 2;                       // items a CTA has in flight
constexpr int kPfAlign = 32;                      // granularity of the virtual positions

struct PrefillArgs {
  void* out;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* q_starts;                        // [num_seqs + 1] first query row (token) each
  unsigned long long* ticket;                     // items drawn; null: one item a CTA at most
  int32_t* status;
  int num_seqs, total_q, num_q_heads, num_kv_heads, group, max_blocks, num_blocks, ctx_cap;
  int window, num_sinks;
  float scale_log2;
};

// One item, as handed to the warps of its CTA.
struct PfItem {
  int seq, kvh;
  int q0;                                         // first token row of the sequence in q, out
  int tok0, ntok;                                 // its new tokens tok0 .. of the sequence
  int pos0;                                       // position of the sequence's first new token
  int ctx, w0;                                    // length; first position its queries' windows reach
  int lo, last;                                   // the item's first window position, last position
  int head, jump;                                 // virtual position v is v (< head) or v + jump
  int tiles;                                      // key tiles; 0: nothing visible
  int end;                                        // no more items
};

template <int D>
struct PfLayout {
  static constexpr int kHalves = D / 64;
  static constexpr int kGroupBytes = kHalves * 1024;           // 8 rows, all halves
  static constexpr int kTileBytes = kHalves * kPfKeys * 128;   // one K or V tile
  static constexpr int kSubBytes = kHalves * kPfSub * 128;     // one subtile of Q
  static constexpr int kSlots = D == 128 ? 4 : 8;              // K and V tiles in flight
  static constexpr int kQOff = kSlots * kTileBytes;
  static constexpr int kOutOff = kQOff + 2 * kSubBytes;        // 4 KB a softmax warp
  static constexpr int kItemOff = kOutOff + 8 * 4096;
  static constexpr int kBarOff = (kItemOff + kPfItems * (int)sizeof(PfItem) + 15) / 16 * 16;
  // kvfull, kvempty [slots]; itemfull, itemempty [items]; sfull, pfull, sfree, pvdone [2]; qfull,
  // qempty, loaded, drain
  static constexpr int kNumBars = 2 * kSlots + 2 * kPfItems + 8 + 4;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;      // tmem base, abort flag
  static constexpr int kBytes = kMiscOff + 16;
  static constexpr int kDynSmem = kBytes + 1024;
  static_assert(kTileBytes % 1024 == 0 && kQOff % 1024 == 0 && kSubBytes % 1024 == 0,
                "128-byte swizzle atoms need 1024-byte alignment");
  static_assert(kDynSmem <= 232448, "one CTA per SM must fit");
};

// Position of virtual position v of an item.
__device__ __forceinline__ int pf_pos(const PfItem& it, int v) {
  return v < it.head ? v : v + it.jump;
}

// x = -inf where `keep` is 0, in place (a conditional expression made the compiler copy every
// score of an unmasked tile too)
__device__ __forceinline__ void mask_to_ninf(uint32_t& x, uint32_t keep) {
  asm("{\n\t.reg .pred p;\n\tsetp.eq.b32 p, %1, 0;\n\t@p mov.b32 %0, 0xff800000;\n\t}"
      : "+r"(x)
      : "r"(keep));
}

// bits r < n (n clamped to 0..32)
__device__ __forceinline__ uint32_t below32(int n) {
  return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}

// Hands out the items of a launch in order, whole warps at a time: the sequences with at least
// one whole item of new tokens in batch order, then the others, whose items are short (a long
// item drawn last is what a launch waits for: 24 ragged chunks 48.2 us against 49.6 in batch
// order alone).  A sequence's items go from its last tokens
// (most positions) to its first, the kv heads of an item's tokens side by side (their CTAs
// read the same block-table entries).
struct PfCursor {
  bool rest = false;             // the sequences with fewer new tokens than an item holds
  long long base = 0;            // first item of the 32 sequences from sbase on
  int sbase = -32;
  long long incl = 0, sum = 0;   // this lane's inclusive item count, all lanes'
  int q0 = 0, n = 0, tiles = 0, ctx = 0;

  __device__ __forceinline__ void load(const PrefillArgs& a, int lane) {
    // (one warp's worth of sequences is still here in the second pass)
    if (!rest || a.num_seqs > 32) {
      const int s = sbase + lane;
      q0 = n = ctx = 0;
      if (s < a.num_seqs) {
        ctx = clamp_ctx(a.context_lens[s], a.ctx_cap, a.status);
        int b = a.q_starts[s], e = a.q_starts[s + 1];
        if (b < 0 || e < b || e > a.total_q) {
          if (a.status) atomicOr(a.status, DEV_BAD_QUERY);
          b = e = 0;
        }
        q0 = b;
        n = e - b;
      }
    }
    const int per = 2 * pf_tokens(a.group);
    tiles = (n < per) == rest ? (n + per - 1) / per : 0;
    incl = (long long)tiles * a.num_kv_heads;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    sum = __shfl_sync(0xffffffffu, incl, 31);
  }
  // item index i (ascending from call to call); every lane of the warp calls it
  __device__ __forceinline__ PfItem find(const PrefillArgs& a, long long i, int lane) {
    PfItem it{};
    while (sbase < 0 || i >= base + sum) {
      if (sbase >= 0) base += sum;
      sbase += 32;
      if (sbase >= a.num_seqs) {
        if (rest) {
          it.end = 1;
          sum = 0;
          return it;
        }
        rest = true;
        sbase = 0;
      }
      load(a, lane);
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, i < base + incl)) - 1;
    const long long first = base + __shfl_sync(0xffffffffu, incl, src) -
                            (long long)__shfl_sync(0xffffffffu, tiles, src) * a.num_kv_heads;
    const int nt = __shfl_sync(0xffffffffu, tiles, src);
    const int nq = __shfl_sync(0xffffffffu, n, src);
    it.q0 = __shfl_sync(0xffffffffu, q0, src);
    it.seq = sbase + src;
    const int j = (int)(i - first);
    it.kvh = j % a.num_kv_heads;
    const int per = 2 * pf_tokens(a.group);
    it.tok0 = (nt - 1 - j / a.num_kv_heads) * per;
    it.ntok = nq - it.tok0 < per ? nq - it.tok0 : per;
    it.ctx = __shfl_sync(0xffffffffu, ctx, src);
    it.pos0 = it.ctx - nq;
    auto win0 = [&](int p) {
      const long long x = (long long)p - a.window + 1;
      return x > 0 ? (int)x : 0;
    };
    it.w0 = win0(it.pos0);
    it.lo = win0(it.pos0 + it.tok0);
    it.last = it.pos0 + it.tok0 + it.ntok - 1;
    if (it.last >= 0) {
      const int ws = it.lo / kPfAlign * kPfAlign;
      const int hs = a.num_sinks < ws ? (a.num_sinks + kPfAlign - 1) / kPfAlign * kPfAlign : ws;
      it.head = hs < ws ? hs : ws;
      it.jump = ws - it.head;
      it.tiles = (it.last + 1 - it.jump + kPfKeys - 1) / kPfKeys;
    }
    return it;
  }
};

template <typename T, int D, int BS>
__global__ void __launch_bounds__(kPfThreads, 1)
    pa_prefill_kernel(const PrefillArgs a, const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv,
                      const __grid_constant__ CUtensorMap tmq) {
  using L = PfLayout<D>;
  constexpr uint32_t kAB = std::is_same_v<T, __nv_bfloat16> ? 1u : 0u;
  // tensor memory: S from column 0, P of subtile j from 128 + 64 j, O from 256 + 128 j
  constexpr uint32_t kPCols = 128, kOCols = 256;
  constexpr int kItemUsers = 8 + 1 + 1 + 1;        // warps that read an item
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sQ = smem + L::kQOff;
  PfItem* items = reinterpret_cast<PfItem*>(smem + L::kItemOff);
  uint64_t* kvfull = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* kvempty = kvfull + L::kSlots;
  uint64_t* itemfull = kvempty + L::kSlots;
  uint64_t* itemempty = itemfull + kPfItems;
  uint64_t* sfull = itemempty + kPfItems;
  uint64_t* pfull = sfull + 2;
  uint64_t* sfree = pfull + 2;
  uint64_t* pvdone = sfree + 2;
  uint64_t* qfull = pvdone + 2;
  uint64_t* qempty = qfull + 1;
  uint64_t* loaded = qempty + 1;
  uint64_t* drain = loaded + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(&kvfull[i], 1);
      mbar_init(&kvempty[i], 1);
    }
    for (int i = 0; i < kPfItems; ++i) {
      mbar_init(&itemfull[i], 1);
      mbar_init(&itemempty[i], kItemUsers);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], kPfSub);
      mbar_init(&pvdone[i], 1);
      mbar_init(&sfree[i], 4);
    }
    mbar_init(qfull, 1);
    mbar_init(qempty, 1);
    mbar_init(loaded, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 32) {
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
    prefetch_tensormap(&tmq);
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  const int Hkv = a.num_kv_heads, group = a.group;
  auto give_up = [&]() {
    if (lane == 0) {
      *abort_flag = 1;
      if (a.status) atomicOr(a.status, DEV_TIMEOUT);
    }
  };
  // (a vote, so that a warp whose lanes disagree at the limit gives up as a whole: what follows
  // a wait is done by whole warps)
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return (bool)__all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort_flag, kWaitLimitNs));
  };
  // whether there is an item k of this CTA (false at the end of the launch or of patience);
  // its fields are read from its slot, which item_done hands back
  auto item_at = [&](int k) {
    const int sl = k % kPfItems;
    if (!wait(&itemfull[sl], (uint32_t)(k / kPfItems) & 1u)) {
      give_up();
      return false;
    }
    return items[sl].end == 0;
  };
  auto item_done = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&itemempty[k % kPfItems]);
  };

  if (warp < 8) {
    // ============================== softmax and output ==============================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int sub = warp >> 2;
    const int r = (warp & 3) * 32 + lane;           // row of the subtile = lane of tensor memory
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + lanes;
    const uint32_t tP = tbase + lanes + kPCols + (uint32_t)(sub * 64);
    const uint32_t tO = tbase + lanes + kOCols + (uint32_t)(sub * 128);
    // a scale of 0 is taken as 1e-37, which gives the same weights (1) and keeps a masked
    // score's -inf * scale from being NaN
    const float sc = fmaxf(fabsf(a.scale_log2), 1e-37f);
    const int tps = pf_tokens(group);
    uint8_t* stage = smem + L::kOutOff + warp * 4096;
    // this thread's query row: new token jr of the subtile, head gr of the group
    const int jr = r / group, gr = r - jr * group;
    uint32_t sph = 0, vph = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!item_at(k)) break;
      const PfItem& it = items[k % kPfItems];
      const int ns = min(it.ntok - sub * tps, tps); // the subtile's tokens
      const bool mine = jr < ns;
      const int token = it.tok0 + sub * tps + jr;
      const bool active = ns > 0 && it.tiles > 0;
      float m = -INFINITY, l = 0.f;
      if (active) {
        auto win0 = [&](int p) {
          const long long x = (long long)p - a.window + 1;
          return x > 0 ? (int)x : 0;
        };
        // this row sees the positions t <= p with t >= plo or t < num_sinks (a row past the
        // item's none)
        const int p = mine ? it.pos0 + token : -1;
        const int plo = win0(p);
        // the subtile's first token sees no position past p_first, its last none before lo_last
        const int p_first = it.pos0 + it.tok0 + sub * tps;
        const int lo_last = win0(p_first + ns - 1);
        const int head = it.head, jump = it.jump, sinks = a.num_sinks, tiles = it.tiles;
        for (int i = 0; i < tiles; ++i) {
          if (!wait(&sfull[sub], sph)) {
            give_up();
            ok = false;
            break;
          }
          sph ^= 1u;
          tc_fence_after();
          uint32_t s[128];
          tmem_ld32(tS, s);
          tmem_ld32(tS + 32, s + 32);
          tmem_ld32(tS + 64, s + 64);
          tmem_ld32(tS + 96, s + 96);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sfree[sub]);
          const int v0 = i * kPfKeys;
          const int t0 = v0 < head ? v0 : v0 + jump;
          // visible whole to every row: one run of positions, none past the first row's own,
          // none before the last row's window (or all of them first tokens)
          const bool whole = (v0 >= head || v0 + kPfKeys <= head) && t0 + kPfKeys - 1 <= p_first &&
                             (t0 >= lo_last || t0 + kPfKeys <= sinks);
          if (!whole) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int v = v0 + 32 * c, t = v < head ? v : v + jump;
              const uint32_t see = below32(p + 1 - t) & (~below32(plo - t) | below32(sinks - t));
#pragma unroll
              for (int j = 0; j < 32; ++j) mask_to_ninf(s[32 * c + j], see & (1u << j));
            }
          }
          float mx[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t* x = s + 32 * c;
            mx[c] = max2_nan(__uint_as_float(x[0]), __uint_as_float(x[1]));
#pragma unroll
            for (int j = 2; j < 32; j += 2)
              mx[c] = max3_nan(mx[c], __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
          }
          const float mt = max2_nan(max3_nan(mx[0], mx[1], mx[2]), mx[3]);
          // a visible score of +inf or NaN makes the row NaN, as the formula's inf - inf does
          // (the weights alone would lose it where they come from the polynomial)
          if (!(mt < INFINITY)) l = NAN;
          // the reference moves on a row's first visible tile and past a gap of 2^8
          const bool move = mt > m && (m == -INFINITY || (mt - m) * sc > kRescaleLog2);
          // the P V of the tile before has read P and is done with O
          if (i > 0) {
            if (!wait(&pvdone[sub], vph)) {
              give_up();
              ok = false;
              break;
            }
            vph ^= 1u;
            tc_fence_after();
          }
          if (__any_sync(0xffffffffu, move)) {
            const float alpha = !move ? 1.f : (m == -INFINITY ? 0.f : ex2((m - mt) * sc));
            if (move) {
              l *= alpha;
              m = mt;
            }
            // O so far is against the old reference; before the first P V there is none
            if (i > 0) {
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                float o[16];
                tmem_ld16(tO + 16 * c, o);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] *= alpha;
                tmem_st16(tO + 16 * c, o);
              }
            }
          }
          const float nms = m == -INFINITY ? 0.f : -m * sc;
          const uint64_t sc2 = pack_f2(sc, sc), nms2 = pack_f2(nms, nms);
          uint64_t ls[2] = {0ull, 0ull};
          // weights of 32 positions: of every 16 pairs kPoly on the FMA units, which a masked
          // tile's -inf must not take (it would leave 2^-126)
          auto weights = [&](int c, auto poly) {
            constexpr int kPoly = decltype(poly)::value;
            float pk[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const uint64_t x = fma_f2(pack_f2(__uint_as_float(s[32 * c + 2 * j]),
                                                __uint_as_float(s[32 * c + 2 * j + 1])),
                                        sc2, nms2);
              float2 w;
              if (j * kPoly / 16 != (j + 1) * kPoly / 16) {
                w = ex2_poly_f2(x);
              } else {
                const float2 y = unpack_f2(x);
                w = make_float2(ex2(y.x), ex2(y.y));
              }
              ls[j & 1] = add_f2(ls[j & 1], pack_f2(w.x, w.y));
              pk[j] = __uint_as_float(pack2<T>(w.x, w.y));
            }
            tmem_st16(tP + 16 * c, pk);
          };
          if (whole) {
#pragma unroll
            for (int c = 0; c < 4; ++c) weights(c, std::integral_constant<int, kPfPoly>{});
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) weights(c, std::integral_constant<int, 0>{});
          }
          const float2 l2 = unpack_f2(add_f2(ls[0], ls[1]));
          l += l2.x + l2.y;
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&pfull[sub]);
        }
        if (ok && !wait(&pvdone[sub], vph)) {
          give_up();
          ok = false;
        }
        if (!ok) break;
        vph ^= 1u;
        tc_fence_after();
        // a row whose scores were all -inf never had a reference: what the polynomial made of
        // them (2^-126) is no weight
        if (m == -INFINITY && l == l) l = 0.f;
      }
      // output rows; a row that sees nothing is zero.  A thread holds a row of O, so 64
      // columns at a time go through the warp's staging area and out as 128 contiguous bytes of
      // each row (a store per thread and row would touch 32 lines an instruction)
      if (ns > 0) {
        const float inv = 1.f / l;
        const int orow = mine ? (it.q0 + token) * a.num_q_heads + it.kvh * group + gr : -1;
        const int u = lane & 7;
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
#pragma unroll 1
          for (int e = 0; e < 2; ++e) {
            uint32_t o[32];
            if (active) {                           // (warp-uniform)
              tmem_ld32(tO + 64 * c + 32 * e, o);
              tmem_wait_ld();
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                w[j] = l == 0.f ? 0u
                                : pack2<T>(__uint_as_float(o[8 * x + 2 * j]) * inv,
                                           __uint_as_float(o[8 * x + 2 * j + 1]) * inv);
              *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * e + x) ^ (lane & 7)) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
#pragma unroll 2
          for (int x = 0; x < 8; ++x) {
            const int rr = x * 4 + (lane >> 3), row = __shfl_sync(0xffffffffu, orow, rr);
            const uint4 w = *reinterpret_cast<const uint4*>(stage + rr * 128 + ((u ^ (rr & 7)) << 4));
            if (row >= 0)
              *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + (long long)row * D + 64 * c + 8 * u) = w;
          }
          __syncwarp();
        }
      }
      tc_fence_before();                            // O is read before the next item's P V
      item_done(k);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8) {
      // ============================== tensor-core issue ==============================
      // The whole warp walks the tiles and one elected lane issues, in branches on elect.sync's
      // own predicate: operands then sit in uniform registers and the instructions follow each
      // other at the tensor cores' pace (64 cycles for 128 x 128 x 16).  Behind a predicate or a
      // branch on the lane number the same instructions took 72 to 100 cycles each to issue.
      const bool one = elect_one();
      const uint32_t idesc_pv = idesc_f16(kAB, 0u, 1u, kPfSub, (uint32_t)D);
      // a negative scale: -Q in its place, so that the softmax may take maxima of scores
      const uint32_t idesc_qk = idesc_f16(kAB, 0u, 0u, kPfSub, kPfKeys) |
                                (a.scale_log2 < 0.f ? kIdescNegateA : 0u);
      const uint64_t dq0 = smem_desc_sw128(smem_u32(sQ), 16u, 1024u);
      const uint64_t dk0 = smem_desc_sw128(smem_u32(smem), 16u, L::kGroupBytes);
      const uint64_t dv0 = smem_desc_sw128(smem_u32(smem), 1024u, L::kGroupBytes);
      constexpr uint32_t kTile16 = L::kTileBytes / 16;
      // slot and phase of the next V tile (fill 1, 3, ..) and the next K tile (0, 2, ..)
      uint32_t sk = 0, kph = 0, sv = 1, vph = 0, qph = 0, pph0 = 0, pph1 = 0, fph0 = 0, fph1 = 0;
      auto next = [](uint32_t& sl, uint32_t& ph) {  // two fills on
        sl += 2;
        if (sl >= (uint32_t)L::kSlots) {
          sl -= (uint32_t)L::kSlots;
          ph ^= 1u;
        }
      };
      auto qk = [&](auto j_) {
        constexpr int j = decltype(j_)::value;
        const uint64_t dk = dk0 + sk * kTile16;
        if (!one) return;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = (ks & 3) * 32;
          tc_mma_f16(tbase,
                     dq0 + ((j * L::kSubBytes + (ks >> 2) * (kPfSub * 128) + off) >> 4),
                     dk + (((ks >> 2) * 1024 + off) >> 4), idesc_qk, ks > 0);
        }
        tc_commit(&sfull[j]);
      };
      auto pv = [&](auto j_, bool more) {
        constexpr int j = decltype(j_)::value;
        const uint64_t dv = dv0 + sv * kTile16;
        if (!one) return;
#pragma unroll
        for (int kk = 0; kk < kPfKeys / 16; ++kk)
          tc_mma_f16_ts(tbase + kOCols + (uint32_t)(j * 128),
                        tbase + kPCols + (uint32_t)(j * 64 + kk * 8),
                        dv + ((kk * 2 * L::kGroupBytes) >> 4), idesc_pv, more || kk > 0);
        tc_commit(&pvdone[j]);
      };
      std::integral_constant<int, 0> A;
      std::integral_constant<int, 1> B;
      bool ok = true;
      for (int k = 0; ok && item_at(k); ++k) {
        const PfItem& it = items[k % kPfItems];
        // (a reduction and a vote, so that the compiler sees one value for the warp)
        const int tiles = __reduce_max_sync(0xffffffffu, it.tiles);
        const bool two = __any_sync(0xffffffffu, it.ntok > pf_tokens(group));
        if (tiles > 0) {
          // Q K^T of subtile j may overwrite S when the softmax has taken the last scores that
          // were put there (the other subtile's, or its own when there is one only)
          auto s_free = [&](int j, uint32_t& ph) {
            const bool x = wait(&sfree[j], ph);
            ph ^= 1u;
            return x;
          };
          ok = wait(qfull, qph) && wait(&kvfull[sk], kph);
          qph ^= 1u;
          if (ok) {
            tc_fence_after();
            qk(A);
            if (two) {
              ok = s_free(0, fph0);
              tc_fence_after();
              if (ok) qk(B);
            }
            if (one) tc_commit(&kvempty[sk]);
            if (tiles == 1 && one) tc_commit(qempty);
            next(sk, kph);
          }
          for (int i = 0; ok && i < tiles; ++i) {
            const bool more = i + 1 < tiles;
            ok = two ? s_free(1, fph1) : s_free(0, fph0);
            if (!ok) break;
            if (more) {
              ok = wait(&kvfull[sk], kph);
              if (!ok) break;
              tc_fence_after();
              qk(A);
            }
            ok = wait(&kvfull[sv], vph) && wait(&pfull[0], pph0);
            if (!ok) break;
            pph0 ^= 1u;
            tc_fence_after();
            pv(A, i > 0);
            if (two) {
              if (more) {
                ok = s_free(0, fph0);
                if (!ok) break;
                tc_fence_after();
                qk(B);
              }
              ok = wait(&pfull[1], pph1);
              if (!ok) break;
              pph1 ^= 1u;
              tc_fence_after();
              pv(B, i > 0);
            }
            if (one) tc_commit(&kvempty[sv]);
            next(sv, vph);
            if (more) {
              if (one) tc_commit(&kvempty[sk]);
              next(sk, kph);
              if (i + 2 == tiles && one) tc_commit(qempty);
            }
          }
          if (!ok) give_up();
        }
        item_done(k);
      }
      // nothing issued here may still run when tensor memory is released
      if (one) {
        tc_commit(drain);
        int no_abort = 0;
        mbar_wait_bounded(drain, 0u, &no_abort, kWaitLimitNs);
      }
      __syncwarp();
    } else if (warp == 9) {
      // ============================== K and V tiles ==============================
      const uint64_t policy = policy_evict_normal();
      const int rows_total = a.num_blocks * Hkv * BS;
      uint32_t f = 0;
      bool ok = true;
      for (int k = 0; ok && item_at(k); ++k) {
        const PfItem it = items[k % kPfItems];
        const int32_t* trow = a.block_tables + (long long)it.seq * a.max_blocks;
        const int S = a.num_sinks;
        // needed by this item; sure: no position of t .. t+n-1 is hidden from every query of
        // the sequence (hidden rows may hold anything)
        auto needed = [&](int t, int n) { return t <= it.last && (t + n > it.lo || t < S); };
        auto sure = [&](int t, int n) { return t + n <= it.ctx && (t >= it.w0 || t + n <= S); };
        auto seen = [&](int t) { return t < it.ctx && (t >= it.w0 || t < S); };
        constexpr int H = BS == 1 ? 1 : (BS < 16 ? BS : 16);   // rows of a TMA box
        constexpr int kBoxes = kPfKeys / H;
        constexpr int kE = BS == 1 ? 4 : 1;                    // table entries a lane holds
        static_assert(kBoxes <= 32 * kE, "one box a lane, or four rows");
        auto entries = [&](int i, int (&e)[kE]) {
#pragma unroll
          for (int x = 0; x < kE; ++x) {
            const int t = pf_pos(it, i * kPfKeys + (x * 32 + lane) * H);
            e[x] = (x * 32 + lane < kBoxes && needed(t, H)) ? __ldg(trow + t / BS) : -1;
          }
        };
        int cur[kE], nxt[kE];
        if (it.tiles) entries(0, cur);
        for (int i = 0; ok && i < it.tiles; ++i) {
          if (i + 1 < it.tiles) entries(i + 1, nxt);
          // row coordinate of the box; out of range (zeros) for a page with a bad id
          int y[kE];
          [[maybe_unused]] bool patch = false;      // its V rows are copied one by one
          bool load_k = false;
#pragma unroll
          for (int x = 0; x < kE; ++x) {
            const int t = pf_pos(it, i * kPfKeys + (x * 32 + lane) * H);
            y[x] = rows_total;
            if (x * 32 + lane < kBoxes && needed(t, H) && (BS != 1 || seen(t))) {
              load_k = true;
              if ((unsigned)cur[x] < (unsigned)a.num_blocks) {
                y[x] = (cur[x] * Hkv + it.kvh) * BS + t % BS;
                patch = BS != 1 && !sure(t, H);
              } else if (a.status) {
                atomicOr(a.status, DEV_BAD_BLOCK_ID);
              }
            }
          }
          for (int kv = 0; ok && kv < 2; ++kv) {
            const int sl = (int)(f % L::kSlots);
            if (!wait(&kvempty[sl], ((f / L::kSlots) & 1u) ^ 1u)) {
              give_up();
              ok = false;
              break;
            }
            ++f;
            uint8_t* dst = smem + sl * L::kTileBytes;
            const CUtensorMap* map = kv ? &tmv : &tmk;
            if constexpr (BS != 1) {
              constexpr int kBoxBytes = H * 128 * L::kHalves;
              // K boxes that nothing needs keep what the slot held (their scores are masked);
              // V boxes become zeros
              const bool box = lane < kBoxes && (kv ? !patch : load_k);
              // rows copied one by one: stored by this warp and fenced against the tensor cores'
              // reads before the tile's barrier is armed (the tensor-core warp would otherwise
              // pay for a fence at every tile)
              unsigned todo = kv ? __ballot_sync(0xffffffffu, patch) : 0u;
              if (todo) {
                while (todo) {
                  const int b = __ffs(todo) - 1;
                  todo &= todo - 1;
                  const int t = pf_pos(it, i * kPfKeys + b * H);
                  const long long yb = __shfl_sync(0xffffffffu, y[0], b);
                  constexpr int CPR = D / 8;        // 16-byte pieces of a row
                  constexpr int kN = H * CPR / 32;
                  uint4 w[kN];
#pragma unroll
                  for (int u = 0; u < kN; ++u) {
                    const int rr = (u * 32 + lane) / CPR, ch = lane % CPR;
                    w[u] = make_uint4(0u, 0u, 0u, 0u);
                    if (seen(t + rr))
                      w[u] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.v_cache) +
                                                             (yb + rr) * D + ch * 8);
                  }
#pragma unroll
                  for (int u = 0; u < kN; ++u) {
                    const int rr = (u * 32 + lane) / CPR, ch = lane % CPR, tr = b * H + rr;
                    *reinterpret_cast<uint4*>(dst + (tr >> 3) * L::kGroupBytes + (ch >> 3) * 1024 +
                                              (tr & 7) * 128 + (((ch & 7) ^ (tr & 7)) << 4)) = w[u];
                  }
                }
                fence_proxy_async_smem();
                __syncwarp();
              }
              const unsigned n = __popc(__ballot_sync(0xffffffffu, box));
              if (lane == 0) mbar_arrive_expect_tx(&kvfull[sl], n * kBoxBytes);
              __syncwarp();
              if (box)
                tma_load_4d(dst + lane * (H / 8) * L::kGroupBytes, map, &kvfull[sl], y[0] >> 3,
                            policy);
            } else {
              // four rows a gather load, one 128-byte half of each
              if (lane == 0) mbar_arrive_expect_tx(&kvfull[sl], L::kTileBytes);
              __syncwarp();
#pragma unroll
              for (int x = 0; x < L::kHalves; ++x) {
                const int e = x * 32 + lane, hf = e % L::kHalves, g = e / L::kHalves;
                int z[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  const int rr = 4 * g + u;         // row of the tile
                  int v[4];
#pragma unroll
                  for (int w = 0; w < 4; ++w) v[w] = __shfl_sync(0xffffffffu, y[w], rr & 31);
                  z[u] = rr < 32 ? v[0] : (rr < 64 ? v[1] : (rr < 96 ? v[2] : v[3]));
                }
                tma_gather4(dst + (g >> 1) * L::kGroupBytes + hf * 1024 + (g & 1) * 512, map,
                            &kvfull[sl], hf * 64, z[0], z[1], z[2], z[3], policy);
              }
            }
          }
#pragma unroll
          for (int x = 0; x < kE; ++x) cur[x] = nxt[x];
        }
        item_done(k);
        if (lane == 0) mbar_arrive(loaded);
      }
      // copies still in flight (only after a failed wait) land before the CTA's memory goes
      if (!ok || *abort_flag) {
        int no_abort = 0;
        for (uint32_t g = f > L::kSlots ? f - L::kSlots : 0; g < f; ++g)
          mbar_wait_bounded(&kvfull[g % L::kSlots], (g / L::kSlots) & 1u, &no_abort, kWaitLimitNs);
      }
    } else if (warp == 10) {
      // ============================== query rows ==============================
      int used = 0;
      for (int k = 0; item_at(k); ++k) {
        const PfItem& it = items[k % kPfItems];
        if (it.tiles > 0) {
          if (used > 0 && !wait(qempty, (uint32_t)(used - 1) & 1u)) {
            give_up();
            break;
          }
          ++used;
          // a subtile's tokens with the heads of this kv head: one box per 64 dims, its rows
          // token-major (tokens behind the sequence's last give rows that nobody writes)
          const int tps = pf_tokens(group), nsub = it.ntok > tps ? 2 : 1;
          if (lane == 0) {
            mbar_arrive_expect_tx(qfull, (uint32_t)(nsub * L::kHalves * tps * group * 128));
            for (int x = 0; x < nsub * L::kHalves; ++x) {
              const int j = x / L::kHalves, hf = x % L::kHalves;
              tma_load_3d(sQ + j * L::kSubBytes + hf * (kPfSub * 128), &tmq, qfull, hf * 64,
                          it.kvh * group, it.q0 + it.tok0 + j * tps);
            }
          }
          __syncwarp();
        }
        item_done(k);
      }
      // a copy still in flight (only after a failed wait) lands before the memory goes
      if (*abort_flag && used > 0) {
        int no_abort = 0;
        mbar_wait_bounded(qfull, (uint32_t)(used - 1) & 1u, &no_abort, kWaitLimitNs);
      }
    } else {
      // ============================== items ==============================
      // The first item is the CTA's index; the later ones are drawn from a counter shared by
      // the launch (zeroed before it), one at a time and late: when every tile of the item
      // before is on its way, so that a CTA does not sit on work while others run dry.  (Drawing
      // two ahead behind short items was no faster: 24 ragged chunks 51.3 us against 48.5.)
      PfCursor cur;
      long long i = blockIdx.x;
      for (int k = 0;; ++k) {
        if (k > 0) {
          // item k - 1 is loaded, and the slot of item k - kPfItems is free
          if (!wait(loaded, (uint32_t)(k - 1) & 1u) ||
              (k >= kPfItems &&
               !wait(&itemempty[k % kPfItems], ((uint32_t)(k / kPfItems) & 1u) ^ 1u))) {
            give_up();
            break;
          }
          // without a counter there are no more items than CTAs
          if (lane == 0)
            i = a.ticket ? (long long)gridDim.x + (long long)atomicAdd(a.ticket, 1ull) : LLONG_MAX;
          i = __shfl_sync(0xffffffffu, i, 0);
        }
        const PfItem it = cur.find(a, i, lane);
        if (lane == 0) {
          items[k % kPfItems] = it;
          mbar_arrive(&itemfull[k % kPfItems]);
        }
        __syncwarp();
        if (it.end) break;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

}  // namespace pkv
