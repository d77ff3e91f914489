// fa_fwd_paged for 17 to 128 rows a sequence (wide groups of query heads,
// drafted tokens, short prompts): the products on the tensor cores' 128-row
// tiles, which cost the same for any number of rows and read each key once.
//
//     S[128 rows x 128 tokens] = Q K^T,   O[128 rows x DV] += P V
// Codes become f16 exactly; a query row is multiplied by a power of two first
// (query_scale: exact down to 2^-31 of its largest value), and the keys' scales,
// one for 16 tokens, multiply the scores.  The values' scales are powers of two too: they go into
// the exponents of the weights, P' = 2^(x - m + k - k0) with k the scale's
// exponent and 2^k0 the unit that O is kept in, rounded to f16.  2^(k0 + 3) is
// the largest scale of the first tile, so a weight under it keeps 11 bits down
// to 2^-17 of the reference and vanishes below 2^-28.  That serves scales between
// 2^(k0-3) and 2^(k0+6); a tile with others ("wide") takes its V as code * 2^(k-k0)
// and its P in bf16, which has the exponents for them.  S, maxima, sums and O
// are fp32.
//
// Work: the tiles of 128 tokens of all sequences and heads form one line that
// is cut into equal pieces, one for each block; cut (sequence, head)s are
// joined by paged_merge_kernel.  Roles of a block (one per SM):
//   warps 0-3   softmax: thread = row = TMEM lane.  The reference of a row
//               follows its maximum when it lags by more than 2^8; so a tile's
//               weights are formed with the reference there is, in one pass
//               over S, and once more in the rare case that it has to move (O
//               is then rescaled in place by the same threads).  Up to 64 or
//               32 rows stand in the 128 lanes twice or four times: each copy
//               takes a half or a quarter of every tile's tokens, with weights
//               of 0 for the others, and the copies are added up at the end.
//   warp 4      issues the MMAs, S of the next tile before P V of this one.
//   warp 5      loads: block table, scales, and the codes by TMA, two tiles ahead.
//   warps 6-13  codes to operands, in the tensor cores' swizzled layout.
// TMEM: S of even and odd tiles, O, P of even and odd tiles.
//
// What bounds it: per 128 tokens and head of 128, 32 KB of codes come in (1300
// cycles at the measured copy rate) and 16 MMAs take 75 cycles each; a tile
// takes about 2600, a chain of load, conversion (700 each of K and V), S (800),
// softmax (1000) and P V (900) with two tiles in flight, whose warps still wait
// for instructions (six roles share the instruction caches) and for TMEM.  Short
// loops were worth more than anything else: the same work unrolled took 90.8 us
// where it takes 70.6.  Starting and ending a (sequence, head) takes 12000
// cycles; counting them as kStart tiles when the line is cut was worth 17 %.
// 16 sequences of 5 new tokens, 32/8 heads of 128, 500 to 8000 keys: 58 us, 2.5
// TB/s of codes; 32 of 32/1 heads: 31 us, of which half is the start and the end;
// 32 x 8000 keys of 2 heads with 64 rows: 57 us, 2.3 TB/s.
#pragma once
#include "fa_paged_attn.cuh"

namespace fa {

template <int DQK, int DV>
struct TcShape {
  static constexpr int kTile = 128, kRows = 128;
  // Tiles that a unit's start and end cost.  us with 3 / 5 / 8, 16 sequences of 5 new tokens and 500 to 8000 keys, 32/8
  // heads: 48.0 / 48.5 / 50.9 at (64, 64), 60.7 / 58.5 / 59.3 at (128, 128), 79.8 / 83.4 / 87.6 at (192, 64), 86.2 / 89.3 /
  // 93.5 at (192, 128), where a tile costs more; 64 sequences of 100 to 600 keys: 44.2 / 41.3 / 41.1, 57.9 / 52.1 / 52.4 and
  // 62.1 / 64.1 / 66.1 at (64, 64), (128, 128) and (192, 128); 32 of 3000 to 9000 keys, 32/1 heads, one token: 25.9 / 24.4 /
  // 25.6, 33.0 / 30.6 / 31.6 and 39.4 / 39.7 / 42.3.  One value within 4.5 % of the best of the three in all.
  static constexpr int kStart = 5;
  static constexpr int kFillWarps = 8, kFillThreads = 32 * kFillWarps;
  static constexpr int kMmaWarp = 4, kLoadWarp = 5, kFillWarp0 = 6;
  static constexpr int kThreads = 32 * (kFillWarp0 + kFillWarps);
  static constexpr int kChunk = 128 * 128;  // 128 rows of 64 operands, swizzled
  static constexpr int kQBytes = DQK / 64 * kChunk;
  // operand slots, K and V tiles by turns: two of each kind, or one where keys are wide.  With three that take turns K
  // of the next tile waits for P V of the one before, and everything behind it too.
  static constexpr int kSlots = DQK == 192 ? 2 : 4;
  static constexpr int kKBytes = DQK / 64 * kChunk, kVBytes = DV / 64 * kChunk;
  static constexpr int kRingBytes = kSlots / 2 * (kKBytes + kVBytes);
  static __device__ __forceinline__ int slot_offset(int slot) {
    return (slot >> 1) * (kKBytes + kVBytes) + (slot & 1) * kKBytes;
  }
  static constexpr int kCodeBytes = kTile * (DQK > DV ? DQK : DV);  // codes of K or V of a tile
  static constexpr int kCodes = 4;                                  // of them under way, K and V by turns
  static constexpr int oRing = kQBytes < 32 * 1024 ? 32 * 1024 : kQBytes, oCodes = oRing + kRingBytes;
  static constexpr int kBytes = oCodes + kCodes * kCodeBytes;  // from a 1024-byte boundary
  static_assert(kBytes + 3 * 1024 <= 227 * 1024, "shared memory, with what the kernel declares itself");
  static_assert(kThreads * 8 <= oRing && 128 * 64 * 4 <= oRing, "the scan of the sequences and sums of copies come there");
  static constexpr uint32_t kColO = 256, kColP = 384;  // TMEM columns (S: 0 and 128)
};

// two e4m3 codes as f16, times a scale, as bf16 (exact)
__device__ __forceinline__ uint32_t scaled_bf16x2(uint32_t f16x2, float scale) {
  const float2 x = f16x2_float2(f16x2);
  return pack_bf16x2(x.x * scale, x.y * scale);
}

__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// 2^k for any k, 0 or infinity beyond fp32
__device__ __forceinline__ float pow2(int k) {
  const float a = __uint_as_float(static_cast<uint32_t>((k >> 1) + 127) << 23);
  return a * __uint_as_float(static_cast<uint32_t>(k - (k >> 1) + 127) << 23);
}

// What the loading warp tells of a tile: its scales, one for 16 tokens, and more.
struct TcTile {
  float ks[8];  // of the keys
  int vk[8];    // of the values: k - k0
  int k0;
  int wide, masked;  // V in bf16; some row does not see all of it
  int left;          // tokens from the tile's first to the sequence's end
};

struct TcParams : PagedParams {
  CUtensorMap tm_k, tm_v;  // (d, token, head, page) of codes; a box is what a tile and a page share
};

template <int DQK, int DV>
__global__ void __launch_bounds__(TcShape<DQK, DV>::kThreads, 1)
    paged_tc_kernel(const __grid_constant__ TcParams p) {
  using L = TcShape<DQK, DV>;
  constexpr int kTile = L::kTile;
  extern __shared__ __align__(1024) uint8_t smem_tc[];
  __shared__ __align__(8) uint64_t bars[2 * L::kSlots + 9 + 2 * L::kCodes];
  __shared__ __align__(16) TcTile tiles[8];  // of eight tiles
  __shared__ uint32_t poison[8][4];       // tokens of a masked tile whose values hold a NaN, for eight tiles
  __shared__ PagedCursor begin_at;
  __shared__ int tile_count;
  __shared__ long long warp_sum[L::kThreads / 32];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t smem0 = smem_u32(smem_tc);
  const uint32_t bar0 = smem_u32(bars);
  auto kv_full = [&](int slot) { return bar0 + 8 * slot; };
  auto kv_empty = [&](int slot) { return bar0 + 8 * (L::kSlots + slot); };
  const uint32_t bar_q = bar0 + 16 * L::kSlots, bar_drain = bar_q + 8, bar_x = bar_q + 16;
  auto s_full = [&](int buf) { return bar_q + 24 + 8 * buf; };
  auto p_full = [&](int buf) { return bar_q + 40 + 8 * buf; };
  // P V of even and odd tiles: with one barrier, whose last phase may still be open when a tile's is waited for, that
  // wait would take the phase before the last for its own
  auto o_full = [&](int buf) { return bar_q + 56 + 8 * buf; };
  auto code_full = [&](int c) { return bar_q + 72 + 8 * c; };
  auto code_empty = [&](int c) { return bar_q + 72 + 8 * (L::kCodes + c); };
  __shared__ float2 copy_ml[128];  // a copy's reference and sum
  const WaitCtx wc{&abort_flag, p.status, p.timeout_ns};

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid < 32) poison[tid >> 2][tid & 3] = 0;
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(kv_full(i), L::kFillWarps);
      mbar_init(kv_empty(i), 1);
    }
    mbar_init(bar_q, 128);
    mbar_init(bar_drain, 1);
    mbar_init(bar_x, 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), 128);
      mbar_init(o_full(i), 1);
    }
    for (int i = 0; i < L::kCodes; ++i) {
      mbar_init(code_full(i), 1);
      mbar_init(code_empty(i), L::kFillWarps);
    }
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  if (warp == L::kMmaWarp) {
    tmem_alloc(smem_u32(&tmem_base), 512);
    tmem_relinquish();
  }

  // ---- the line of tiles, as in paged_attn_kernel with one team a block ----
  PagedLine line;
  paged_line<kTile, L::kThreads, 1, L::kStart>(p, reinterpret_cast<long long*>(smem_tc), warp_sum, &begin_at, &tile_count,
                                               line);
  const int count = tile_count;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;

  // first token that some row of the sequence does not see
  auto least_limit = [&](const PagedSeq& s) {
    if (!p.causal) return s.len;
    const int l = s.len - s.n + 1;
    return l < 0 ? 0 : l < s.len ? l : s.len;
  };

  if (count > 0) {
    if (warp < 4) {
      // ======== softmax ========
      PagedCursor cur = begin_at;
      const long long piece = line.piece(0);
      const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp * 32) << 16);
      const uint32_t t_o = t_lane + L::kColO;
      // lanes' copies of the rows: this thread's row, and the tokens of a tile that its copy takes
      const int copies = 1 << p.copy_shift, copy_rows = 128 >> p.copy_shift, copy = tid >> (7 - p.copy_shift);
      const int r = tid & (copy_rows - 1);
      const int groups = 8 >> p.copy_shift, group0 = copy * groups;  // of 16 tokens
      float fac = 0.f, ref = -INFINITY, sum = 0.f;
      int limit = 0, min_limit = 0, unit_k0 = 0, x_phase = 0;
      bool started_here = false;
      bool ok = true;
      for (int i = 0; i < count && ok; ++i) {
        const bool first = i == 0 || cur.tile == 0;
        const bool active = warp * 32 - copy * copy_rows < cur.s.rows;  // some row of this warp is one of the sequence's
        if (first) {
          started_here = cur.tile == 0;
          // this thread's query row as f16, its largest value at the top of the range, by way of its place;
          // eight lanes fetch 128 bytes of a row
          const int pos = r / p.ratio;
          const uint32_t at = smem0 + tid * 128;
          auto column = [&](int c) { return at + (c >> 3) * L::kChunk + (((c & 7) ^ (tid & 7)) << 4); };
          uint32_t top = 0;  // exponents of two columns
          const int64_t row_at =
              (static_cast<int64_t>(cur.s.cu0 + pos) * p.heads_q + cur.head * p.ratio + (r - pos * p.ratio)) * DQK;
#pragma unroll 1
          for (int k = 0; k < 32; k += 4) {
            const int from = k + (lane >> 3), there = __shfl_sync(0xffffffffu, r, from);
            const __nv_bfloat16* src = p.q + __shfl_sync(0xffffffffu, row_at, from) + 8 * (lane & 7);
            const uint32_t dst = smem0 + (warp * 32 + from) * 128 + (((lane & 7) ^ (from & 7)) << 4);
            if (there < cur.s.rows) {
#pragma unroll
              for (int c = 0; c < DQK / 64; ++c) cp_async16(dst + c * L::kChunk, src + 64 * c);
            }
          }
          cp_async_commit();
          cp_async_wait<0>();
          __syncwarp();
          if (r < cur.s.rows) {
#pragma unroll 4
            for (int c = 0; c < DQK / 8; ++c) {
              const uint4 x = lds128(column(c));
              top = __vmaxu2(__vmaxu2(top, x.x & 0x7f807f80u), x.y & 0x7f807f80u);
              top = __vmaxu2(__vmaxu2(top, x.z & 0x7f807f80u), x.w & 0x7f807f80u);
            }
          }
          const QueryScale qs =
              query_scale(static_cast<int>(((top & 0xffffu) > (top >> 16) ? top & 0xffffu : top >> 16) >> 7));
          const float down = qs.down;
          fac = p.scale_log2 * qs.up;
#pragma unroll 4
          for (int c = 0; c < DQK / 8; ++c) {
            const uint4 x = r < cur.s.rows ? lds128(column(c)) : make_uint4(0, 0, 0, 0);
            auto half = [&](uint32_t w) {
              return pack_f16x2(__uint_as_float(w << 16) * down, __uint_as_float(w & 0xffff0000u) * down);
            };
            sts128(column(c), make_uint4(half(x.x), half(x.y), half(x.z), half(x.w)));
          }
          ref = -INFINITY;
          sum = 0.f;
          min_limit = least_limit(cur.s);
          limit = cur.s.len;
          if (p.causal && r < cur.s.rows) {
            limit = cur.s.len - cur.s.n + pos + 1;
            limit = limit < 0 ? 0 : limit > cur.s.len ? cur.s.len : limit;
          }
          fence_proxy_async_smem();
          mbar_arrive(bar_q);
          if (i == 0 && copies > 1) {  // weights of other copies' tokens are 0 for good
            uint32_t zero[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) zero[k] = 0;
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) tmem_st32(t_lane + L::kColP + c, zero);
            tmem_wait_st();
          }
        }
        const int buf = i & 1, token0 = cur.tile * kTile;
        const bool masked = token0 + kTile > min_limit;
        ok = __all_sync(0xffffffffu, tc_wait(s_full(buf), (i >> 1) & 1, wc));
        if (masked && ok) {  // which of the tile's values are no numbers is known once they are converted
          const int e = 2 * i + 1;
          ok = __all_sync(0xffffffffu, tc_wait(kv_full(e % L::kSlots), (e / L::kSlots) & 1, wc));
        }
        if (!ok) break;
        tc_fence_after();
        if (first) unit_k0 = tiles[i & 7].k0;
        if (active) {
          const uint32_t t_s = t_lane + 128 * buf, t_p = t_lane + L::kColP + 64 * buf;
          const bool wide = tiles[i & 7].wide != 0;
          float mx = -INFINITY, part = 0.f;
          // weights of the tile with the present reference, their sum, and the scores' maximum
          auto weights = [&](auto with_mask) {
            constexpr bool kMask = decltype(with_mask)::value;
            const float back = ref == -INFINITY ? 0.f : -ref;
            mx = -INFINITY;
            part = 0.f;
#pragma unroll 1
            for (int g = group0; g < group0 + groups; ++g) {
              uint32_t s[16];
              tmem_ld16_wait(t_s + 16 * g, s);
              const int vk = tiles[i & 7].vk[g];
              const float f = fac * tiles[i & 7].ks[g];
              const float from = wide ? back : back + static_cast<float>(vk);
              const uint32_t bad = kMask ? poison[i & 7][g >> 1] >> (16 * (g & 1)) : 0u;
              const int left = kMask ? limit - token0 - 16 * g : 16;  // columns that the row sees
              float m = -INFINITY, e0 = 0.f, e1 = 0.f;
#pragma unroll
              for (int c = 0; c < 16; c += 2) {
                if (kMask) {
                  if (c < left) m = fmaxf(m, __uint_as_float(s[c]));
                  if (c + 1 < left) m = fmaxf(m, __uint_as_float(s[c + 1]));
                } else {
                  m = fmax3(m, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
                }
              }
              if (m != -INFINITY) mx = fmaxf(mx, m * f);
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                float e = ex2_approx(fmaf(__uint_as_float(s[c]), f, from));
                if (kMask) {
                  if ((bad >> c) & 1) e = __uint_as_float(0x7fc00000u);
                  if (c >= left) e = 0.f;
                }
                if (c & 1) e1 += e;
                else e0 += e;
                s[c] = __float_as_uint(e);
              }
              part = wide ? part + (e0 + e1) : fmaf(e0 + e1, pow2(-vk), part);
              uint32_t pk[8];
              if (wide) {
#pragma unroll
                for (int c = 0; c < 8; ++c) pk[c] = pack_bf16x2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]));
              } else {
#pragma unroll
                for (int c = 0; c < 8; ++c) pk[c] = pack_f16x2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]));
              }
              tmem_st8(t_p + 8 * g, pk);
            }
          };
          for (;;) {
            if (masked) weights(std::true_type{});
            else weights(std::false_type{});
            const bool move = mx > ref + kRefLag;  // also from -inf
            if (!__any_sync(0xffffffffu, move)) break;
            const float alpha = move ? ex2_approx(ref - mx) : 1.f;
            if (move) ref = mx;
            sum *= alpha;
            if (!first) {
              // P V of the tile before has to be in O
              ok = __all_sync(0xffffffffu, tc_wait(o_full(buf ^ 1), ((i - 1) >> 1) & 1, wc));
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < DV; c += 32) {
                uint32_t v[32];
                tmem_ld32_wait(t_o + c, v);
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
                tmem_st32(t_o + c, v);
              }
            }
            tmem_wait_st();  // also of the first weights, which are written again
          }
          if (!ok) break;
          sum += part;
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(p_full(buf));

        const bool unit_end = cur.tile + 1 == cur.s.tiles;
        if (unit_end || i + 1 == count) {
          const bool whole = started_here && unit_end;
          if (!whole && started_here && tid == 0) {
            PagedJoin j;
            j.last = static_cast<int>((cur.at + (cur.s.tiles - 1 - cur.tile)) / line.per);
            j.cu0 = cur.s.cu0;
            j.head = cur.head;
            j.rows = cur.s.rows;
            p.part.joins[piece] = j;
          }
          ok = __all_sync(0xffffffffu, tc_wait(o_full(buf), (i >> 1) & 1, wc));
          if (!ok) break;
          tc_fence_after();
          auto meet = [&]() {  // all softmax threads
            mbar_arrive(bar_x);
            return __all_sync(0xffffffffu, tc_wait(bar_x, x_phase++ & 1, wc));
          };
          // A value that is no number makes its whole row so, here as where its tile is masked.  (A lane of no weight
          // saw none: its O is not looked at.)
          bool nan = false;
#pragma unroll 1
          for (int c = 0; c < DV; c += 32) {
            uint32_t v[32];
            tmem_ld32_wait(t_o + c, v);
#pragma unroll
            for (int k = 0; k < 32; ++k) nan |= isnan(__uint_as_float(v[k]));
          }
          if (nan && sum != 0.f) sum = __uint_as_float(0x7fc00000u);
          const float rf = sum != 0.f && ref == -INFINITY ? 0.f : ref;
          const int64_t part = 2 * piece + (started_here ? 1 : 0);
          float top = rf, l = sum;
          if (copies > 1) {
            copy_ml[tid] = make_float2(rf, sum);
            ok = meet();
            if (!ok) break;
            for (int k = 0; k < copies; ++k) top = fmaxf(top, copy_ml[k * copy_rows + r].x);
          }
          const float base = top == -INFINITY ? 0.f : top;
          if (copies > 1) {
            l = 0.f;
            for (int k = 0; k < copies; ++k) {
              const float2 ml = copy_ml[k * copy_rows + r];
              l = fmaf(ex2_approx(ml.x - base), ml.y, l);
            }
          }
          const float unit = pow2(unit_k0);
          const float scale = ex2_approx(rf - base) * (!whole ? unit : l == 0.f ? 0.f : unit / l);
          if (copy == 0 && r < cur.s.rows) {
            if (!whole) {
              p.part.ml[part * L::kRows + r] = make_float2(top + kPShift, l);
            } else if (p.lse != nullptr) {
              const int pos = r / p.ratio;
              p.lse[static_cast<int64_t>(cur.head * p.ratio + (r - pos * p.ratio)) * p.total_q + cur.s.cu0 + pos] =
                  l == 0.f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
            }
          }
          // All lanes' O goes through the queries' place in shared memory, which the MMAs are done with, 64 columns at
          // a time in 16-byte steps that spread over the banks; half a warp then takes a row, adds up its copies and
          // writes 64 columns side by side.  A lane of no weight (a row without a key) multiplied nothing: its O is
          // whatever P V of zeros left.
          const int step = lane & 15;
#pragma unroll 1
          for (int c0 = 0; c0 < DV && ok; c0 += 64) {
#pragma unroll 1
            for (int c = 0; c < 64; c += 16) {
              uint32_t v[16];
              tmem_ld16_wait(t_o + c0 + c, v);
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] = scale == 0.f ? 0u : __float_as_uint(__uint_as_float(v[k]) * scale);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                sts128(smem0 + tid * 256 + (((c / 4 + k) ^ (tid & 15)) << 4),
                       make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]));
            }
            ok = meet();
            if (!ok) break;
#pragma unroll 1
            for (int row = 2 * warp + (lane >> 4); row < cur.s.rows; row += 8) {
              auto lane_o = [&](int k) {
                const int from = k * copy_rows + row;
                const uint4 y = lds128(smem0 + from * 256 + ((step ^ (from & 15)) << 4));
                return make_float4(__uint_as_float(y.x), __uint_as_float(y.y), __uint_as_float(y.z), __uint_as_float(y.w));
              };
              float4 v = lane_o(0);
              for (int k = 1; k < copies; ++k) {
                const float4 y = lane_o(k);
                v = make_float4(v.x + y.x, v.y + y.y, v.z + y.z, v.w + y.w);
              }
              const int c = c0 + 4 * step;
              if (whole) {
                const int pos = row / p.ratio, hq = cur.head * p.ratio + (row - pos * p.ratio);
                *reinterpret_cast<uint2*>(p.o + (static_cast<int64_t>(cur.s.cu0 + pos) * p.heads_q + hq) * DV + c) =
                    make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
              } else {
                *reinterpret_cast<float4*>(p.part.o + (part * L::kRows + row) * DV + c) = v;
              }
            }
            ok = meet();  // read before the next columns or queries come there
          }
          if (!ok) break;
        }
        if (i + 1 < count) paged_next<kTile, L::kStart>(p, cur);
      }
    } else if (warp == L::kLoadWarp) {
      // ======== loads ========
      PagedCursor cur = begin_at;
      int page0 = 0, entry = 0, k0 = 0;  // lane l holds the table's entry of page page0 + l
      auto load_pages = [&](int first_page) {
        page0 = first_page;
        entry = 0;
        if (((first_page + lane) << p.page_shift) < cur.s.len) {
          entry = p.table[cur.b * p.table_stride + first_page + lane];
          if (entry < 0 || entry >= p.num_pages) {
            paged_error(p.status, kSitePagedPage, cur.b);
            entry = 0;
          }
        }
      };
      // what is known of a tile before its copies are due: each lane's page, and the scales, lane l's of the tokens
      // 16 (l % 8) ..
      struct Ahead {
        int entry, head, left, ek, ev;
        int box;  // this lane's copy in the tile, or -1
        bool first, masked;
      };
      auto look_ahead = [&](bool first_of_piece) {
        Ahead a;
        const int token0 = cur.tile * kTile;
        a.left = cur.s.len - token0;
        a.head = cur.head;
        a.first = first_of_piece || cur.tile == 0;
        a.masked = token0 + kTile > least_limit(cur.s);
        int boxes = (a.left + (1 << p.page_shift) - 1) >> p.page_shift;
        if (boxes > (kTile >> p.page_shift)) boxes = kTile >> p.page_shift;
        const int first = (token0 >> p.page_shift) - page0;
        a.box = lane >= first && lane - first < boxes ? lane - first : -1;
        a.entry = entry;
        const int group = lane & 7;
        const int e = __shfl_sync(0xffffffffu, entry, (first + ((16 * group) >> p.page_shift)) & 31);
        a.ek = a.ev = 0;
        if (16 * group < a.left) {
          const int64_t at = static_cast<int64_t>(e) * p.heads_kv + cur.head;
          a.ek = p.k_scale[at];
          a.ev = p.v_scale[at];
        }
        return a;
      };
      auto advance = [&]() {
        const int b = cur.b, head = cur.head;
        paged_next<kTile, L::kStart>(p, cur);
        const int page = (cur.tile * kTile) >> p.page_shift;
        if (cur.b != b || (cur.head != head && page0 != 0) || page + kTile / 16 > page0 + 32) load_pages(page);
      };
      // what the other warps read of a tile
      auto tell = [&](int i, const Ahead& a) {
        // the unit of O: 2^-3 of the largest of the values' scales in the piece's first tile of the sequence, kept
        // moderate; a scale that is NaN makes the keys' NaN
        const bool none = 16 * (lane & 7) >= a.left, nan = !none && a.ev == 255;
        int vk = none || nan ? -1000 : a.ev - 127;
        if (a.first) {
          k0 = __reduce_max_sync(0xffffffffu, vk);
          k0 = k0 == -1000 ? 0 : k0 - 3;
          k0 = k0 < -20 ? -20 : k0 > 30 ? 30 : k0;
        }
        vk = none || nan ? 0 : vk - k0;
        const bool wide = __any_sync(0xffffffffu, vk < -3 || vk > 6);
        TcTile& t = tiles[i & 7];
        if (lane < 8) {
          t.ks[lane] = none ? 1.f : scale_of(nan ? 255 : a.ek);
          t.vk[lane] = vk;
        }
        if (lane == 0) {
          t.k0 = k0;
          t.wide = wide;
          t.masked = a.masked;
          t.left = a.left;
        }
      };
      load_pages((cur.tile * kTile) >> p.page_shift);
      Ahead now = look_ahead(true);
      // an entry's codes: even ones K, odd ones V; each copy announces its own bytes
      auto place_free = [&](int e) {
        const int place = e % L::kCodes, use = e / L::kCodes;
        return use == 0 || __all_sync(0xffffffffu, tc_wait(code_empty(place), (use - 1) & 1, wc));
      };
      auto announce = [&](int e, int d) {
        asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(code_full(e % L::kCodes)),
                     "r"(d << p.page_shift)
                     : "memory");
        return smem0 + L::oCodes + (e % L::kCodes) * L::kCodeBytes;
      };
      int issued = 0;
      for (int i = 0; i < count; ++i) {
        if (!place_free(2 * i)) break;
        const uint32_t row = now.box << p.page_shift;
        if (now.box >= 0) {
          const uint32_t dst = announce(2 * i, DQK), full = code_full((2 * i) % L::kCodes);
          if constexpr (DQK == 128) {
            tma_load_4d(dst + row * 128, &p.tm_k, full, 0, 0, now.head, now.entry);
          } else {
#pragma unroll
            for (int c = 0; c < DQK / 64; ++c)
              tma_load_4d(dst + c * kTile * 64 + row * 64, &p.tm_k, full, 64 * c, 0, now.head, now.entry);
          }
        }
        tell(i, now);
        __syncwarp();
        if (lane == 0) mbar_arrive(code_full((2 * i) % L::kCodes));
        ++issued;
        if (!place_free(2 * i + 1)) break;
        if (now.box >= 0)
          tma_load_4d(announce(2 * i + 1, DV) + row * DV, &p.tm_v, code_full((2 * i + 1) % L::kCodes), 0, 0, now.head,
                      now.entry);
        __syncwarp();
        if (lane == 0) mbar_arrive(code_full((2 * i + 1) % L::kCodes));
        ++issued;
        if (i + 1 < count) {
          advance();
          now = look_ahead(false);
        }
      }
      // the copies under way land before the block's memory is given up, also after a failure
      const uint64_t t0 = globaltimer_ns();
      for (int e = issued > L::kCodes ? issued - L::kCodes : 0; e < issued; ++e)
        while (!mbar_try_wait(code_full(e % L::kCodes), (e / L::kCodes) & 1) && globaltimer_ns() - t0 < 1000000000ull) {
        }
    } else if (warp >= L::kFillWarp0) {
      // ======== codes to operands ========
      const int ft = tid - 32 * L::kFillWarp0;
      // Eight lanes take 4 neighbouring chunks of 16 codes of the rows r and r ^ 5 (so that they read and write
      // different banks); a thread takes a column group of the rows my_row and my_row + 64 at a time.
      const int pair = (ft >> 3) & 3, low = (ft >> 2) & 1;
      const int my_row = ((ft >> 5) << 3) + (low ? pair ^ 5 : pair), my_chunk = ft & 3;
      // where a chunk's codes lie (128-byte rows: column groups side by side; 64-byte rows: one after the other),
      // and where the two halves of its operands go in a column group's 128 rows
      const uint32_t at128 = my_row * 128 + ((my_chunk ^ (my_row & 7)) << 4);
      const uint32_t at64 = my_row * 64 + ((my_chunk ^ ((my_row >> 1) & 3)) << 4);
      auto code_at = [&](int d, int group, int half) -> uint32_t {
        return d == 128 ? (at128 ^ (group << 6)) + half * (64 * 128) : at64 + group * (kTile * 64) + half * (64 * 64);
      };
      const uint32_t out0 = my_row * 128 + (((2 * my_chunk) ^ (my_row & 7)) << 4);
      const uint32_t out1 = my_row * 128 + (((2 * my_chunk + 1) ^ (my_row & 7)) << 4);
      auto to_f16 = [&](uint32_t from, uint32_t (&f)[8]) {
        const uint4 v = lds128(from);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          f[2 * x] = e4m3x2_f16x2(w[x]);
          f[2 * x + 1] = e4m3x2_hi_f16x2(w[x]);
        }
      };
      auto put = [&](uint32_t at, const uint32_t (&f)[8]) {
        sts128(at + out0, make_uint4(f[0], f[1], f[2], f[3]));
        sts128(at + out1, make_uint4(f[4], f[5], f[6], f[7]));
      };
      // an entry's slot of the ring is free once the MMA on its last use is done
      auto slot_free = [&](int e) {
        const int slot = e % L::kSlots, use = e / L::kSlots;
        return use == 0 || __all_sync(0xffffffffu, tc_wait(kv_empty(slot), (use - 1) & 1, wc));
      };
      auto slot_done = [&](int e) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(kv_full(e % L::kSlots));
          mbar_arrive(code_empty(e % L::kCodes));
        }
      };
      // an entry's codes, or 0 after a failure
      auto codes_of = [&](int e) -> uint32_t {
        const int place = e % L::kCodes;
        if (!__all_sync(0xffffffffu, tc_wait(code_full(place), (e / L::kCodes) & 1, wc)) || !slot_free(e)) return 0;
        return smem0 + L::oCodes + place * L::kCodeBytes;
      };
      // One short loop for K and V: what bounds this kernel more than anything else is the fetching of instructions.
      for (int e = 0; e < 2 * count; ++e) {
        const uint32_t codes = codes_of(e);
        if (codes == 0) break;
        const int i = e >> 1, d = e & 1 ? DV : DQK;
        const uint32_t to = smem0 + L::oRing + L::slot_offset(e % L::kSlots);
        if ((e & 1) && tiles[i & 7].masked != 0) {  // hidden from some row: no value may be NaN (own chunks, in place)
          const int left = tiles[i & 7].left;
#pragma unroll 1
          for (int k = 0; k < 2 * (DV / 64); ++k) {
            const int row = my_row + 64 * (k & 1);
            const uint32_t at = codes + code_at(DV, k >> 1, k & 1);
            uint4 v = lds128(at);
            uint32_t* w = &v.x;
            const bool inside = row < left;
            uint32_t any = 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t bad = ((w[x] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
              any |= bad;
              w[x] = inside ? w[x] & ~((bad >> 7) * 0xffu) : 0u;
            }
            if (any != 0 && inside) atomicOr(&poison[i & 7][row >> 5], 1u << (row & 31));
            sts128(at, v);
          }
        }
        // cleared for a tile far enough ahead that neither its conversion has begun nor the softmax of the
        // last tile that used these words is still under way
        if ((e & 1) && ft < 4) poison[(i + 4) & 7][ft] = 0;
        if (!(e & 1) || tiles[i & 7].wide == 0) {
#pragma unroll 1
          for (int c = 0; c < d / 64; ++c) {
            uint32_t f[2][8];
            to_f16(codes + code_at(d, c, 0), f[0]);
            to_f16(codes + code_at(d, c, 1), f[1]);
            put(to + c * L::kChunk, f[0]);
            put(to + c * L::kChunk + 64 * 128, f[1]);
          }
        } else {
#pragma unroll 1
          for (int k = 0; k < 2 * (DV / 64); ++k) {
            const float scale = pow2(tiles[i & 7].vk[(my_row + 64 * (k & 1)) >> 4]);
            uint32_t f[8];
            to_f16(codes + code_at(DV, k >> 1, k & 1), f);
#pragma unroll
            for (int x = 0; x < 8; ++x) f[x] = scaled_bf16x2(f[x], scale);
            put(to + (k >> 1) * L::kChunk + (k & 1) * 64 * 128, f);
          }
        }
        slot_done(e);
      }
    } else {
      // ======== MMA ========
      constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false, false) & ~((1u << 7) | (1u << 10));  // f16 operands
      constexpr uint32_t kIdescWide = idesc_bf16_f32(128, DV, false, true);  // bf16 operands
      constexpr uint32_t kIdescO = kIdescWide & ~((1u << 7) | (1u << 10));
      const uint32_t leader = lane == 0 ? 1u : 0u;
      // what the instructions take comes by a shuffle, which tells the compiler that it is the same in all lanes
      auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
      const uint32_t t0_mem = uniform(tmem), base = uniform(smem0);
      const int n = uniform(count);
      auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, tc_wait(bar, parity, wc)); };
      auto wait_entry = [&](int e) { return wait(kv_full(e % L::kSlots), (e / L::kSlots) & 1); };
      auto issue_s = [&](int i) {  // S of tile i; its K slot is free after it
        const int slot = (2 * i) % L::kSlots;
        const uint32_t k_at = base + L::oRing + L::slot_offset(slot);
#pragma unroll 1
        for (int c = 0; c < DQK / 64; ++c) {
          const uint32_t co = opaque_u32(static_cast<uint32_t>(c * L::kChunk));
          mma_ss_x4<2, 2>(t0_mem + 128 * (i & 1), smem_desc_sw128(base + co, 16, 1024), smem_desc_sw128(k_at + co, 16, 1024),
                          kIdescS, c != 0 ? 1u : 0u, leader);
        }
        mma_commit(s_full(i & 1), leader);
        mma_commit(kv_empty(slot), leader);
      };
      PagedCursor cur = begin_at;
      int tile = uniform(cur.tile), unit_tiles = uniform(cur.s.tiles), units = 0;
      bool ok = true;
      for (int i = 0; i < n && ok; ++i) {
        if (i == 0 || tile == 0) {
          ok = wait(bar_q, units & 1) && wait_entry(2 * i);
          if (!ok) break;
          ++units;
          tc_fence_after();
          issue_s(i);
        }
        if (tile + 1 < unit_tiles && i + 1 < n) {  // the unit goes on
          ok = wait_entry(2 * i + 2);
          if (!ok) break;
          tc_fence_after();
          issue_s(i + 1);
        }
        ok = wait(p_full(i & 1), (i >> 1) & 1) && wait_entry(2 * i + 1);
        if (!ok) break;
        tc_fence_after();
        const int slot = (2 * i + 1) % L::kSlots;
        const uint32_t v_at = base + L::oRing + L::slot_offset(slot);
        const uint32_t begun = i != 0 && tile != 0 ? 1u : 0u;  // O holds tiles of this unit
        const uint32_t p_at = t0_mem + L::kColP + 64 * (i & 1);
        const uint32_t idesc = uniform(tiles[i & 7].wide) == 0 ? kIdescO : kIdescWide;
#pragma unroll 1
        for (int h = 0; h < 2; ++h)
          mma_ts_x4<(16 * 128 >> 4)>(t0_mem + L::kColO, p_at + 32 * h,
                                     smem_desc_sw128(v_at + static_cast<uint32_t>(h * 64 * 128), L::kChunk, 1024), idesc,
                                     h != 0 ? 1u : begun, leader);
        mma_commit(o_full(i & 1), leader);
        mma_commit(kv_empty(slot), leader);
        if (++tile == unit_tiles && i + 1 < n) {
          cur.tile = cur.s.tiles - 1;
          paged_next<kTile, L::kStart>(p, cur);
          tile = 0;
          unit_tiles = uniform(cur.s.tiles);
        }
      }
      // every MMA issued so far has completed once this fires
      mma_commit(bar_drain, leader);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(bar_drain, 0))
        if (globaltimer_ns() - t0 > p.timeout_ns) {
          raise_abort(wc, kStatusTimeout, kSitePagedWait);
          break;
        }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == L::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (p.after) asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace fa
