// fa_fwd_paged for 17 to 128 rows a sequence (wide groups of query heads,
// drafted tokens, short prompts): the products on the tensor cores' 128-row
// tiles, which cost the same for any number of rows and read each key once.
//
//     S[128 rows x 128 tokens] = Q K^T,   O[128 rows x DV] += P V
// Codes become f16 exactly; a query row is divided by a power of two first (f16
// then holds its bf16 values), and the keys' scales, one for 16 tokens,
// multiply the scores.  The values' scales are powers of two too: they go into
// the exponents of the weights, P' = 2^(x - m + k - k0) with k the scale's
// exponent and 2^k0 the unit that O is kept in, rounded to f16.  That holds for
// scales between 2^(k0-3) and 2^(k0+6) (weights then lose bits only below
// 2^-11 of the largest, vanish below 2^-21); a tile with others ("wide") takes its
// V as code * 2^(k-k0) and its P in bf16, which has the exponents for them.
// S, maxima, sums and O are fp32.
//
// Work: the tiles of 128 tokens of all sequences and heads form one line that
// is cut into equal pieces, one for each block; cut (sequence, head)s are
// joined by paged_merge_kernel.  Roles of a block (one per SM):
//   warps 0-3   softmax: thread = row = TMEM lane.  The reference of a row
//               follows its maximum when it lags by more than 2^8; so a tile's
//               weights are formed with the reference there is, in one pass
//               over S, and once more in the rare case that it has to move (O
//               is then rescaled in place by the same threads).
//   warp 4      issues the MMAs, S of the next tile before P V of this one.
//   warps 5-12  codes to operands: each thread copies its 16-byte chunks to
//               shared memory two tiles ahead, converts them and writes them
//               in the tensor cores' swizzled layout.
// TMEM: S of even and odd tiles, O, P of even and odd tiles.  What bounds it:
// per 128 tokens and head 32 KB of codes come in (about 1400 cycles at this
// GPU's bandwidth), the two products take about 1000 cycles, the exponentials
// of a warp of rows 1024, the shared memory carries 230 KB (1800 cycles), and
// the conversion issues about 600 instructions a scheduler.
#pragma once
#include "fa_paged_attn.cuh"

namespace fa {

template <int DQK, int DV>
struct TcShape {
  static constexpr int kTile = 128, kRows = 128;
  static constexpr int kFillWarps = 8, kFillThreads = 32 * kFillWarps;
  static constexpr int kMmaWarp = 4, kFillWarp0 = 5;
  static constexpr int kThreads = 32 * (kFillWarp0 + kFillWarps);
  static constexpr int kChunk = 128 * 128;  // 128 rows of 64 operands, swizzled
  static constexpr int kQBytes = DQK / 64 * kChunk;
  // operand slots, K and V tiles by turns: three, or with wide keys one of each kind
  static constexpr int kSlots = DQK == 192 ? 2 : 3;
  static constexpr int kKBytes = DQK / 64 * kChunk, kVBytes = DV / 64 * kChunk;
  static constexpr int kRingBytes = kSlots == 3 ? 3 * kKBytes : kKBytes + kVBytes;
  static __device__ __forceinline__ int slot_offset(int slot) { return slot * kKBytes; }
  static constexpr int kCodeBytes = kTile * (DQK + DV);  // codes of a tile
  static constexpr int kCodes = 2;                       // tiles under way
  static constexpr int oRing = kQBytes, oCodes = oRing + kRingBytes;
  static constexpr int kBytes = oCodes + kCodes * kCodeBytes + 1024;
  static_assert(kBytes <= 227 * 1024 - 10 * 1024, "shared memory");
  static constexpr uint32_t kColO = 256, kColP = 384;  // TMEM columns (S: 0 and 128)
};

// two e4m3 codes as f16, times a scale, as bf16 (exact)
__device__ __forceinline__ uint32_t scaled_bf16x2(uint32_t f16x2, float scale) {
  const float2 x = f16x2_float2(f16x2);
  return pack_bf16x2(x.x * scale, x.y * scale);
}

// 2^k for any k, 0 or infinity beyond fp32
__device__ __forceinline__ float pow2(int k) {
  const float a = __uint_as_float(static_cast<uint32_t>((k >> 1) + 127) << 23);
  return a * __uint_as_float(static_cast<uint32_t>(k - (k >> 1) + 127) << 23);
}

// What the roles know of a tile's scales, one for 16 tokens.
struct TcTile {
  float ks[8];   // of the keys
  int vk[8];     // of the values: k - k0
  int wide, k0;
};

template <int DQK, int DV>
__global__ void __launch_bounds__(TcShape<DQK, DV>::kThreads, 1)
    paged_tc_kernel(const __grid_constant__ PagedParams p) {
  using L = TcShape<DQK, DV>;
  constexpr int kTile = L::kTile;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * L::kSlots + 7];
  __shared__ __align__(16) TcTile tiles[4];  // of four tiles
  __shared__ uint32_t poison[8][4];       // tokens of a masked tile whose values hold a NaN, for eight tiles
  __shared__ PagedCursor begin_at;
  __shared__ long long scan[L::kThreads];
  __shared__ long long warp_sum[L::kThreads / 32];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t smem0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_u32(bars);
  auto kv_full = [&](int slot) { return bar0 + 8 * slot; };
  auto kv_empty = [&](int slot) { return bar0 + 8 * (L::kSlots + slot); };
  const uint32_t bar_q = bar0 + 16 * L::kSlots, bar_o = bar_q + 8, bar_drain = bar_q + 16;
  auto s_full = [&](int buf) { return bar_q + 24 + 8 * buf; };
  auto p_full = [&](int buf) { return bar_q + 40 + 8 * buf; };
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
    mbar_init(bar_o, 1);
    mbar_init(bar_drain, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), 128);
    }
    fence_mbar_init();
  }
  if (warp == L::kMmaWarp) {
    tmem_alloc(smem_u32(&tmem_base), 512);
    tmem_relinquish();
  }

  // ---- the line of tiles, as in paged_attn_kernel with one team a block ----
  PagedLine line;
  paged_line<kTile, L::kThreads, 1>(p, scan, warp_sum, &begin_at, line);
  const int count = line.count(0);
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
      const int r = tid;
      float fac = 0.f, ref = -INFINITY, sum = 0.f;
      int limit = 0, min_limit = 0, unit_k0 = 0;
      bool started_here = false;
      bool ok = true;
      for (int i = 0; i < count && ok; ++i) {
        const bool first = i == 0 || cur.tile == 0;
        const bool active = warp * 32 < cur.s.rows;  // some row of this warp is one of the sequence's
        if (first) {
          started_here = cur.tile == 0;
          // this thread's query row as f16, divided by the power of two of its largest value
          uint4 raw[DQK / 8];
          const int pos = r / p.ratio;
          if (r < cur.s.rows) {
            const __nv_bfloat16* src =
                p.q + (static_cast<int64_t>(cur.s.cu0 + pos) * p.heads_q + cur.head * p.ratio + (r - pos * p.ratio)) * DQK;
#pragma unroll
            for (int c = 0; c < DQK / 8; ++c) raw[c] = __ldg(reinterpret_cast<const uint4*>(src) + c);
          } else {
#pragma unroll
            for (int c = 0; c < DQK / 8; ++c) raw[c] = make_uint4(0, 0, 0, 0);
          }
          uint32_t top = 0;
#pragma unroll
          for (int c = 0; c < DQK / 8; ++c) {
            const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t a = w[k] & 0x7f80u, b = (w[k] >> 16) & 0x7f80u;
              top = top > a ? top : a;
              top = top > b ? top : b;
            }
          }
          int ex = static_cast<int>(top >> 7);
          ex = ex == 0 || ex == 255 ? 127 : ex;  // a row of zeros, or one that holds no numbers
          const float down = scale_of(254 - ex);
          fac = p.scale_log2 * scale_of(ex);
          ref = -INFINITY;
          sum = 0.f;
          min_limit = least_limit(cur.s);
          limit = cur.s.len;
          if (p.causal && r < cur.s.rows) {
            limit = cur.s.len - cur.s.n + pos + 1;
            limit = limit < 0 ? 0 : limit > cur.s.len ? cur.s.len : limit;
          }
#pragma unroll
          for (int c = 0; c < DQK / 8; ++c) {
            const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
            uint32_t f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              f[k] = pack_f16x2(__uint_as_float(w[k] << 16) * down, __uint_as_float(w[k] & 0xffff0000u) * down);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             smem0 + (c >> 3) * L::kChunk + r * 128 + (((c & 7) ^ (r & 7)) << 4)),
                         "r"(f[0]), "r"(f[1]), "r"(f[2]), "r"(f[3])
                         : "memory");
          }
          fence_proxy_async_smem();
          mbar_arrive(bar_q);
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
        if (active) {
          const uint32_t t_s = t_lane + 128 * buf, t_p = t_lane + L::kColP + 64 * buf;
          const bool wide = tiles[i & 3].wide != 0;
          if (first) unit_k0 = tiles[i & 3].k0;
          float mx = -INFINITY, part = 0.f;
          // weights of the tile with the present reference, their sum, and the scores' maximum
          auto weights = [&](auto with_mask) {
            constexpr bool kMask = decltype(with_mask)::value;
            const float back = ref == -INFINITY ? 0.f : -ref;
            mx = -INFINITY;
            part = 0.f;
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {
              uint32_t s[32];
              tmem_ld32_wait(t_s + 32 * g, s);
              const float2 ks = *reinterpret_cast<const float2*>(&tiles[i & 3].ks[2 * g]);
              const int2 vk = *reinterpret_cast<const int2*>(&tiles[i & 3].vk[2 * g]);
              const float f0 = fac * ks.x, f1 = fac * ks.y;
              const float back0 = wide ? back : back + static_cast<float>(vk.x);
              const float back1 = wide ? back : back + static_cast<float>(vk.y);
              float e0 = 0.f, e1 = 0.f;
              const uint32_t bad = kMask ? poison[i & 7][g] : 0u;
              const int left = kMask ? limit - token0 - 32 * g : 32;  // columns that the row sees
              float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
              for (int c = 0; c < 16; c += 2) {
                if (kMask) {
                  if (c < left) m0 = fmaxf(m0, __uint_as_float(s[c]));
                  if (c + 1 < left) m0 = fmaxf(m0, __uint_as_float(s[c + 1]));
                  if (c + 16 < left) m1 = fmaxf(m1, __uint_as_float(s[c + 16]));
                  if (c + 17 < left) m1 = fmaxf(m1, __uint_as_float(s[c + 17]));
                } else {
                  m0 = fmax3(m0, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
                  m1 = fmax3(m1, __uint_as_float(s[c + 16]), __uint_as_float(s[c + 17]));
                }
              }
              if (m0 != -INFINITY) mx = fmaxf(mx, m0 * f0);
              if (m1 != -INFINITY) mx = fmaxf(mx, m1 * f1);
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                float e = ex2_approx(fmaf(__uint_as_float(s[c]), c < 16 ? f0 : f1, c < 16 ? back0 : back1));
                if (kMask) {
                  if ((bad >> c) & 1) e = __uint_as_float(0x7fc00000u);
                  if (c >= left) e = 0.f;
                }
                if (c < 16) e0 += e;
                else e1 += e;
                s[c] = __float_as_uint(e);
              }
              part += wide ? e0 + e1 : fmaf(e0, pow2(-vk.x), e1 * pow2(-vk.y));
              uint32_t pk[16];
              if (wide) {
#pragma unroll
                for (int c = 0; c < 16; ++c) pk[c] = pack_bf16x2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]));
              } else {
#pragma unroll
                for (int c = 0; c < 16; ++c) pk[c] = pack_f16x2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]));
              }
              tmem_st16(t_p + 16 * g, pk);
            }
          };
          if (masked) weights(std::true_type{});
          else weights(std::false_type{});
          const bool move = mx > ref + kRefLag;  // also from -inf
          if (__any_sync(0xffffffffu, move)) {
            const float alpha = move ? ex2_approx(ref - mx) : 1.f;
            if (move) ref = mx;
            sum *= alpha;
            if (!first) {
              // P V of the tile before has to be in O
              ok = __all_sync(0xffffffffu, tc_wait(bar_o, (i - 1) & 1, wc));
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
            if (masked) weights(std::true_type{});
            else weights(std::false_type{});
          }
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
            j.last = static_cast<int>((piece * line.per + i + (cur.s.tiles - 1 - cur.tile)) / line.per);
            j.cu0 = cur.s.cu0;
            j.head = cur.head;
            j.rows = cur.s.rows;
            p.joins[piece] = j;
          }
          ok = __all_sync(0xffffffffu, tc_wait(bar_o, i & 1, wc));
          if (!ok) break;
          tc_fence_after();
          if (active) {
            const int64_t part = 2 * piece + (started_here ? 1 : 0);
            const int pos = r / p.ratio, hq = cur.head * p.ratio + (r - pos * p.ratio);
            const int64_t token = cur.s.cu0 + pos;
            const float rf = sum != 0.f && ref == -INFINITY ? 0.f : ref;
            const float unit = pow2(unit_k0);
            const float inv = sum == 0.f ? 0.f : unit / sum;
#pragma unroll 1
            for (int c = 0; c < DV; c += 32) {
              uint32_t v[32];
              tmem_ld32_wait(t_o + c, v);
              if (r < cur.s.rows) {
                if (whole) {
                  uint4* dst = reinterpret_cast<uint4*>(p.o + (token * p.heads_q + hq) * DV + c);
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    uint32_t w[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                      w[x] = pack_bf16x2(__uint_as_float(v[8 * k + 2 * x]) * inv, __uint_as_float(v[8 * k + 2 * x + 1]) * inv);
                    // a row without a key multiplied nothing: its O is whatever P V of zeros left
                    dst[k] = sum == 0.f ? make_uint4(0, 0, 0, 0) : make_uint4(w[0], w[1], w[2], w[3]);
                  }
                } else {
                  uint4* dst = reinterpret_cast<uint4*>(p.part_o + (part * L::kRows + r) * DV + c);
#pragma unroll
                  for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * unit);
#pragma unroll
                  for (int k = 0; k < 8; ++k) dst[k] = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                }
              }
            }
            if (r < cur.s.rows) {
              if (!whole) p.part_ml[part * L::kRows + r] = make_float2(rf + kPShift, sum);
              else if (p.lse != nullptr)
                p.lse[hq * p.total_q + token] = sum == 0.f ? -INFINITY : (rf + log2f(sum)) * 0.6931471805599453f;
            }
          }
        }
        if (i + 1 < count) paged_next<kTile>(p, cur);
      }
    } else if (warp >= L::kFillWarp0) {
      // ======== codes to operands ========
      const int ft = tid - 32 * L::kFillWarp0;
      PagedCursor ahead = begin_at, cur = begin_at;  // the tiles that are copied and converted next
      int copied = 0;                                // tiles under way or done
      int page0 = 0, entry = 0;
      auto load_pages = [&](int first_page) {
        page0 = first_page;
        entry = 0;
        if (((first_page + lane) << p.page_shift) < ahead.s.len) {
          entry = p.table[ahead.b * p.table_stride + first_page + lane];
          if (entry < 0 || entry >= p.num_pages) {
            paged_error(p.status, kSitePagedPage, ahead.b);
            entry = 0;
          }
        }
      };
      load_pages((ahead.tile * kTile) >> p.page_shift);
      // Eight lanes take 4 neighbouring chunks of 16 codes of two neighbouring rows (so that they write to
      // different banks); pass k of a thread is column group k % (D / 64) of row my_row or my_row + 64.
      const int my_row = 2 * (ft >> 3) + ((ft >> 2) & 1), my_chunk = ft & 3;
      // where the two halves of a chunk's operands go in a column group's 128 rows
      const uint32_t out0 = my_row * 128 + (((2 * my_chunk) ^ (my_row & 7)) << 4);
      const uint32_t out1 = my_row * 128 + (((2 * my_chunk + 1) ^ (my_row & 7)) << 4);
      constexpr int kPassK = 2 * (DQK / 64), kPassV = 2 * (DV / 64);
      constexpr uint32_t kPassBytes = L::kFillThreads * 16;  // of codes
      // The next tile's codes, and in lanes 0 .. 7 its scales, one for 16 tokens.
      int ek = 127, ev = 127, ek_next = 127, ev_next = 127;
      auto fetch = [&]() {
        ek_next = ev_next = 127;
        if (copied < count) {
          const uint32_t dst = smem0 + L::oCodes + (copied & 1) * L::kCodeBytes + ft * 16;
          const int token0 = ahead.tile * kTile, mask = (1 << p.page_shift) - 1;
          const uint8_t* kh = p.k + ahead.head * p.k_head + my_chunk * 16;
          const uint8_t* vh = p.v + ahead.head * p.v_head + my_chunk * 16;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int t = token0 + my_row + 64 * h;
            const int e = __shfl_sync(0xffffffffu, entry, ((t >> p.page_shift) - page0) & 31);
            if (t < ahead.s.len) {
              const uint32_t in_page = t & mask;
              const uint8_t* ks = kh + e * p.k_page + static_cast<uint64_t>(in_page * p.k_token);
              const uint8_t* vs = vh + e * p.v_page + static_cast<uint64_t>(in_page * p.v_token);
#pragma unroll
              for (int k = 0; k < DQK / 64; ++k) cp_async16(dst + (h * (DQK / 64) + k) * kPassBytes, ks + 64 * k);
#pragma unroll
              for (int k = 0; k < DV / 64; ++k) cp_async16(dst + (kPassK + h * (DV / 64) + k) * kPassBytes, vs + 64 * k);
            }
          }
          const int token = token0 + 16 * (lane & 7);
          const int e = __shfl_sync(0xffffffffu, entry, ((token >> p.page_shift) - page0) & 31);
          if (token < ahead.s.len) {
            const int64_t at = static_cast<int64_t>(e) * p.heads_kv + ahead.head;
            ek_next = p.k_scale[at];
            ev_next = p.v_scale[at];
          } else {
            ev_next = -1;  // no tokens: does not count
          }
          if (copied + 1 < count) {
            const int b = ahead.b, head = ahead.head;
            paged_next<kTile>(p, ahead);
            const int next = (ahead.tile * kTile) >> p.page_shift;
            if (ahead.b != b || (ahead.head != head && page0 != 0) || next + kTile / 16 > page0 + 32) load_pages(next);
          }
        }
        ++copied;
        cp_async_commit();  // a group for each tile, empty ones at the end
      };
      fetch();
      ek = ek_next, ev = ev_next;
      fetch();
      bool ok = true;
      int k0 = 0;
      for (int i = 0; i < count && ok; ++i) {
        const int token0 = cur.tile * kTile;
        const bool masked = token0 + kTile > least_limit(cur.s);
        // the unit of O: 2^-3 of the largest of the values' scales in the piece's first tile of the sequence, kept
        // moderate; a scale that is NaN makes the keys' NaN
        const bool none = ev < 0, nan = ev == 255;
        int vk = none || nan ? -1000 : ev - 127;
        if (i == 0 || cur.tile == 0) {
          k0 = __reduce_max_sync(0xffffffffu, vk);
          k0 = k0 == -1000 ? 0 : k0 - 3;
          k0 = k0 < -20 ? -20 : k0 > 30 ? 30 : k0;
        }
        vk = none || nan ? 0 : vk - k0;
        const bool wide = __any_sync(0xffffffffu, vk < -3 || vk > 6);
        const float ks = nan ? scale_of(255) : scale_of(ek);
        cp_async_wait<1>();
        const uint32_t codes = smem0 + L::oCodes + (i & 1) * L::kCodeBytes + ft * 16;
        // an entry's slot of the ring is free once the MMA on its last use is done
        auto slot_free = [&](int e) {
          const int slot = e % L::kSlots, use = e / L::kSlots;
          return use == 0 || __all_sync(0xffffffffu, tc_wait(kv_empty(slot), (use - 1) & 1, wc));
        };
        auto slot_done = [&](int e) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(kv_full(e % L::kSlots));
        };
        auto put = [&](uint32_t at, const uint32_t (&f)[8]) {
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + out0), "r"(f[0]), "r"(f[1]), "r"(f[2]),
                       "r"(f[3])
                       : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + out1), "r"(f[4]), "r"(f[5]), "r"(f[6]),
                       "r"(f[7])
                       : "memory");
        };
        auto to_f16 = [&](const uint4& v, uint32_t (&f)[8]) {
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            f[2 * x] = e4m3x2_f16x2(w[x]);
            f[2 * x + 1] = e4m3x2_hi_f16x2(w[x]);
          }
        };

        if (!slot_free(2 * i)) break;
        if (ft < 8) {
          tiles[i & 3].ks[ft] = ks;
          tiles[i & 3].vk[ft] = vk;
          if (ft == 0) tiles[i & 3].wide = wide, tiles[i & 3].k0 = k0;
        }
        {
          const uint32_t tile = smem0 + L::oRing + L::slot_offset((2 * i) % L::kSlots);
#pragma unroll
          for (int k = 0; k < kPassK; ++k) {
            uint32_t f[8];
            to_f16(lds128(codes + k * kPassBytes), f);
            put(tile + (k % (DQK / 64)) * L::kChunk + (k / (DQK / 64)) * 64 * 128, f);
          }
        }
        slot_done(2 * i);

        const uint32_t v_codes = codes + kPassK * kPassBytes;
        if (masked) {  // hidden from some row: no value may be NaN
#pragma unroll 1
          for (int k = 0; k < kPassV; ++k) {
            const int row = my_row + 64 * (k / (DV / 64));
            uint4 v = lds128(v_codes + k * kPassBytes);
            uint32_t* w = &v.x;
            const bool inside = token0 + row < cur.s.len;
            uint32_t any = 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t bad = ((w[x] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
              any |= bad;
              w[x] = inside ? w[x] & ~((bad >> 7) * 0xffu) : 0u;
            }
            if (any != 0 && inside) atomicOr(&poison[i & 7][row >> 5], 1u << (row & 31));
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(v_codes + k * kPassBytes), "r"(v.x), "r"(v.y),
                         "r"(v.z), "r"(v.w)
                         : "memory");
          }
        }
        if (!slot_free(2 * i + 1)) break;
        // cleared for a tile far enough ahead that neither its conversion has begun nor the softmax of the
        // last tile that used these words is still under way
        if (ft < 4) poison[(i + 4) & 7][ft] = 0;
        {
          const uint32_t tile = smem0 + L::oRing + L::slot_offset((2 * i + 1) % L::kSlots);
          if (!wide) {
#pragma unroll
            for (int k = 0; k < kPassV; ++k) {
              uint32_t f[8];
              to_f16(lds128(v_codes + k * kPassBytes), f);
              put(tile + (k % (DV / 64)) * L::kChunk + (k / (DV / 64)) * 64 * 128, f);
            }
          } else {
#pragma unroll 1
            for (int k = 0; k < kPassV; ++k) {
              const int row = my_row + 64 * (k / (DV / 64));
              const float scale = pow2(__shfl_sync(0xffffffffu, vk, row >> 4));
              uint32_t f[8];
              to_f16(lds128(v_codes + k * kPassBytes), f);
#pragma unroll
              for (int x = 0; x < 8; ++x) f[x] = scaled_bf16x2(f[x], scale);
              put(tile + (k % (DV / 64)) * L::kChunk + (k / (DV / 64)) * 64 * 128, f);
            }
          }
        }
        slot_done(2 * i + 1);
        ek = ek_next, ev = ev_next;
        fetch();
        if (i + 1 < count) paged_next<kTile>(p, cur);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
      // ======== MMA ========
      constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false, false) & ~((1u << 7) | (1u << 10));  // f16 operands
      constexpr uint32_t kIdescWide = idesc_bf16_f32(128, DV, false, true);  // bf16 operands
      constexpr uint32_t kIdescO = kIdescWide & ~((1u << 7) | (1u << 10));
      const uint32_t leader = lane == 0 ? 1u : 0u;
      auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, tc_wait(bar, parity, wc)); };
      auto wait_entry = [&](int e) { return wait(kv_full(e % L::kSlots), (e / L::kSlots) & 1); };
      auto issue_s = [&](int i) {  // S of tile i; its K slot is free after it
        const int slot = (2 * i) % L::kSlots;
        const uint32_t k_at = smem0 + L::oRing + L::slot_offset(slot);
#pragma unroll
        for (int c = 0; c < DQK / 64; ++c) {
          const uint32_t co = opaque_u32(static_cast<uint32_t>(c * L::kChunk));
          mma_ss_x4<2, 2>(tmem + 128 * (i & 1), smem_desc_sw128(smem0 + co, 16, 1024), smem_desc_sw128(k_at + co, 16, 1024),
                          kIdescS, c != 0 ? 1u : 0u, leader);
        }
        mma_commit(s_full(i & 1), leader);
        mma_commit(kv_empty(slot), leader);
      };
      PagedCursor cur = begin_at;
      int units = 0;
      bool ok = true;
      for (int i = 0; i < count && ok; ++i) {
        if (i == 0 || cur.tile == 0) {
          ok = wait(bar_q, units & 1) && wait_entry(2 * i);
          if (!ok) break;
          ++units;
          tc_fence_after();
          issue_s(i);
        }
        const bool more = cur.tile + 1 < cur.s.tiles && i + 1 < count;  // the unit goes on
        if (more) {
          ok = wait_entry(2 * i + 2);
          if (!ok) break;
          tc_fence_after();
          issue_s(i + 1);
        }
        ok = wait(p_full(i & 1), (i >> 1) & 1) && wait_entry(2 * i + 1);
        if (!ok) break;
        tc_fence_after();
        const int slot = (2 * i + 1) % L::kSlots;
        const uint32_t v_at = smem0 + L::oRing + L::slot_offset(slot);
        const bool begun = i != 0 && cur.tile != 0;  // O holds tiles of this unit
        const uint32_t idesc = tiles[i & 3].wide != 0 ? kIdescWide : kIdescO;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t va = opaque_u32(v_at + static_cast<uint32_t>(h * 64 * 128));
          mma_ts_x4<(16 * 128 >> 4)>(tmem + L::kColO, tmem + L::kColP + 64 * (i & 1) + 32 * h, smem_desc_sw128(va, L::kChunk, 1024),
                                     idesc, h != 0 || begun ? 1u : 0u, leader);
        }
        mma_commit(bar_o, leader);
        mma_commit(kv_empty(slot), leader);
        if (i + 1 < count) paged_next<kTile>(p, cur);
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
}

}  // namespace fa
