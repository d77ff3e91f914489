// fa_fwd_paged for 17 to 128 rows a sequence (wide groups of query heads,
// drafted tokens, short prompts): the products on the tensor cores' 128-row
// tiles, which cost the same for any number of rows and read each key once.
//
//     S[128 rows x 128 tokens] = Q K^T,   O[128 rows x DV] += P V
// K codes become f16 exactly; a query row is divided by a power of two first
// (f16 then holds its bf16 values), and the keys' scales, one for 16 tokens,
// multiply the scores.  V codes times their scales are bf16 numbers exactly;
// P is rounded to bf16 for that product.  S, maxima, sums and O are fp32.
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
//   warps 5-20  codes to operands: each thread copies its 16-byte chunks to
//               shared memory two tiles ahead, converts them and writes them
//               in the tensor cores' swizzled layout.
// TMEM: S of even and odd tiles, O, P of even and odd tiles.  What bounds it:
// per 128 tokens and head 32 KB of codes come in (about 1400 cycles at this
// GPU's bandwidth), the two products take about 1000 cycles, the exponentials
// of a warp of rows 1024, the shared memory carries 230 KB (1800 cycles), and
// the conversion issues about 1200 instructions a scheduler.
#pragma once
#include "fa_paged_attn.cuh"

namespace fa {

template <int DQK, int DV>
struct TcShape {
  static constexpr int kTile = 128, kRows = 128;
  static constexpr int kFillWarps = 16, kFillThreads = 32 * kFillWarps;
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

template <int DQK, int DV>
__global__ void __launch_bounds__(TcShape<DQK, DV>::kThreads, 1)
    paged_tc_kernel(const __grid_constant__ PagedParams p) {
  using L = TcShape<DQK, DV>;
  constexpr int kTile = L::kTile;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * L::kSlots + 7];
  __shared__ float k_scales[4][8];        // of a tile's 16-token groups, for four tiles
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
      int limit = 0, min_limit = 0;
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
          float mx = -INFINITY, part = 0.f;
          // weights of the tile with the present reference, their sum, and the scores' maximum
          auto weights = [&](auto with_mask) {
            constexpr bool kMask = decltype(with_mask)::value;
            const float back = ref == -INFINITY ? 0.f : -ref;
            float e0 = 0.f, e1 = 0.f;
            mx = -INFINITY;
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {
              uint32_t s[32];
              tmem_ld32_wait(t_s + 32 * g, s);
              const float2 ks = *reinterpret_cast<const float2*>(&k_scales[i & 3][2 * g]);
              const float f0 = fac * ks.x, f1 = fac * ks.y;
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
              uint32_t pk[16];
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                const float f = c < 16 ? f0 : f1;
                float a = ex2_approx(fmaf(__uint_as_float(s[c]), f, back));
                float b = ex2_approx(fmaf(__uint_as_float(s[c + 1]), f, back));
                if (kMask) {
                  if ((bad >> c) & 1) a = __uint_as_float(0x7fc00000u);
                  if ((bad >> (c + 1)) & 1) b = __uint_as_float(0x7fc00000u);
                  if (c >= left) a = 0.f;
                  if (c + 1 >= left) b = 0.f;
                }
                e0 += a;
                e1 += b;
                pk[c / 2] = pack_bf16x2(a, b);
              }
              tmem_st16(t_p + 16 * g, pk);
            }
            part = e0 + e1;
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
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
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
      // this thread's chunks of a tile's K or V: row and 16-code column of chunk number k
      auto copy = [&](auto is_k, uint32_t dst) {
        constexpr bool kK = decltype(is_k)::value;
        constexpr int D = kK ? DQK : DV, kChunks = D / 16, kPer = kTile * kChunks / L::kFillThreads;
        const uint8_t* base = kK ? p.k + ahead.head * p.k_head : p.v + ahead.head * p.v_head;
        const int64_t page_stride = kK ? p.k_page : p.v_page;
        const uint32_t ts = kK ? p.k_token : p.v_token;
        const int token0 = ahead.tile * kTile;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const int at = k * L::kFillThreads + ft, row = at / kChunks, chunk = at % kChunks;
          const int t = token0 + row;
          const int e = __shfl_sync(0xffffffffu, entry, ((t >> p.page_shift) - page0) & 31);
          if (t < ahead.s.len)
            cp_async16(dst + k * L::kFillThreads * 16,
                       base + e * page_stride + static_cast<uint32_t>(t & ((1 << p.page_shift) - 1)) * ts + chunk * 16);
        }
      };
      // The next tile's codes, and in lanes 0 .. 7 its scales, one for 16 tokens.
      int ek = 127, ev = 127, ek_next = 127, ev_next = 127;
      auto fetch = [&]() {
        ek_next = ev_next = 127;
        if (copied < count) {
          const uint32_t dst = smem0 + L::oCodes + (copied & 1) * L::kCodeBytes + ft * 16;
          copy(std::true_type{}, dst);
          copy(std::false_type{}, dst + kTile * DQK);
          const int token = ahead.tile * kTile + 16 * (lane & 7);
          const int e = __shfl_sync(0xffffffffu, entry, ((token >> p.page_shift) - page0) & 31);
          if (lane < 8 && token < ahead.s.len) {
            const int64_t at = static_cast<int64_t>(e) * p.heads_kv + ahead.head;
            ek_next = p.k_scale[at];
            ev_next = p.v_scale[at];
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
      for (int i = 0; i < count && ok; ++i) {
        const int token0 = cur.tile * kTile;
        const bool masked = token0 + kTile > least_limit(cur.s);
        cp_async_wait<1>();
        const uint32_t codes = smem0 + L::oCodes + (i & 1) * L::kCodeBytes + ft * 16;
        const float ks = ev == 255 ? scale_of(255) : scale_of(ek);  // NaN in either: NaN scores
        const float vs = ev == 255 ? 1.f : scale_of(ev);
        auto convert = [&](auto kind, uint32_t from, uint32_t tile) {
          constexpr bool kK = decltype(kind)::value;
          constexpr int D = kK ? DQK : DV, kChunks = D / 16, kPer = kTile * kChunks / L::kFillThreads;
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            const int at = k * L::kFillThreads + ft, row = at / kChunks, chunk = at % kChunks;
            const float scale = kK ? 1.f : __shfl_sync(0xffffffffu, vs, row >> 4);
            const uint4 v = lds128(from + k * L::kFillThreads * 16);
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
            if (!kK && masked) {  // hidden from some row: no value may be NaN
              const bool inside = token0 + row < cur.s.len;
              uint32_t any = 0;
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint32_t nan = ((w[x] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                any |= nan;
                w[x] = inside ? w[x] & ~((nan >> 7) * 0xffu) : 0u;
              }
              if (any != 0 && inside) atomicOr(&poison[i & 7][row >> 5], 1u << (row & 31));
            }
            uint32_t f[8];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              f[2 * x] = e4m3x2_f16x2(w[x]);
              f[2 * x + 1] = e4m3x2_hi_f16x2(w[x]);
              if constexpr (!kK) {
                f[2 * x] = scaled_bf16x2(f[2 * x], scale);
                f[2 * x + 1] = scaled_bf16x2(f[2 * x + 1], scale);
              }
            }
            // two groups of 8 operands; lanes of the right half write their second first (banks)
            const uint32_t line_at = tile + (chunk >> 2) * L::kChunk + row * 128;
            const int c0 = (2 * chunk) & 7;
            const bool swap = kChunks == 8 && (chunk & 4) != 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const bool second = (h == 1) != swap;
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                               line_at + (((c0 + (second ? 1 : 0)) ^ (row & 7)) << 4)),
                           "r"(second ? f[4] : f[0]), "r"(second ? f[5] : f[1]), "r"(second ? f[6] : f[2]),
                           "r"(second ? f[7] : f[3])
                           : "memory");
            }
          }
        };
        // entry 2 i (K) and 2 i + 1 (V) of the ring: free once the MMA on its last use is done
        auto put = [&](auto kind, int e, uint32_t from) -> bool {
          const int slot = e % L::kSlots, use = e / L::kSlots;
          if (use > 0 && !__all_sync(0xffffffffu, tc_wait(kv_empty(slot), (use - 1) & 1, wc))) return false;
          if (decltype(kind)::value) {
            if (ft < 8) k_scales[i & 3][ft] = ks;
          } else if (ft < 4) {
            // cleared for a tile far enough ahead that neither its conversion has begun nor the softmax of the
            // last tile that used these words is still under way
            poison[(i + 4) & 7][ft] = 0;
          }
          convert(kind, from, smem0 + L::oRing + L::slot_offset(slot));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(kv_full(slot));
          return true;
        };
        ok = put(std::true_type{}, 2 * i, codes) && put(std::false_type{}, 2 * i + 1, codes + kTile * DQK);
        if (!ok) break;
        ek = ek_next, ev = ev_next;
        fetch();
        if (i + 1 < count) paged_next<kTile>(p, cur);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
      // ======== MMA ========
      constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false, false) & ~((1u << 7) | (1u << 10));  // f16 operands
      constexpr uint32_t kIdescO = idesc_bf16_f32(128, DV, false, true);
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
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t va = opaque_u32(v_at + static_cast<uint32_t>(h * 64 * 128));
          mma_ts_x4<(16 * 128 >> 4)>(tmem + L::kColO, tmem + L::kColP + 64 * (i & 1) + 32 * h, smem_desc_sw128(va, L::kChunk, 1024),
                                     kIdescO, h != 0 || begun ? 1u : 0u, leader);
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
