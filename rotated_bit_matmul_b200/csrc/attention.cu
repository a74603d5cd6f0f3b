// Attention of one new token per sequence over a paged key-value cache.
//
//   o_h = sum_j p_j v_j,  p = softmax_j(scale q_h . k_j),  j in [max(0, len - window), len),
//   query head h reading key head h / (n_heads / n_kv). A sequence without keys gives zeros.
//
// The cache is read once, so HBM bounds the work: the query heads of one key head are the
// rows of one 16-row matrix tile, and both products run on mma.sync m16n8k16 (a few percent
// of its rate; the 128-row tcgen05 tile would be filled to an eighth or less by one token's
// heads). Softmax statistics and outputs are fp32 with a running maximum.
//
// Split. The tiles of 64 keys of all (sequence, key head) pairs form one line, which is cut
// into equal shares, one per CTA, from the lengths on the device: any mix of lengths is
// balanced without the host knowing it, and a captured launch stays valid as lengths grow.
// A pair that lies in one share is finished there. One that is cut leaves an fp32 partial
// (maximum, sum, unnormalised output) per share in the workspace, and join_kernel adds them
// in the order of the keys, so results do not depend on timing.
//
// Inside a CTA each of four warps owns 16 keys of every tile and everything it needs for
// them: it looks up the pages, copies K and V rows with cp.async into its own ring of
// stages, and keeps its own maximum, sum and output. The loop has no CTA barrier; the warps
// meet only where a pair ends. Rows outside the mask are not read: their bytes in shared
// memory are zero-filled, so what a page holds behind a sequence's end (NaN included) has
// no effect. The copies run ahead across pair borders, so the ring stays full.
//
// The probabilities enter the second product as hi + lo halves of the cache's type (two
// products into one accumulator): a single bf16 p would add an error of 2^-9 per key, as
// large as the rounding of the output itself.
#include "serve.cuh"
#include "serve.h"

namespace harp {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 64;   // keys per tile; 16 per warp
constexpr int kRows = 16;   // query heads per tile
constexpr int kMaxCtas = 2 * 148;
constexpr int kJoinThreads = 128;
constexpr int kJoinRows = 4;  // heads per CTA of the join

struct Params {
  AttnCall c;
  int group;       // query heads per key head
  int hblocks;     // tiles of kRows query heads per key head
  int units;       // n_kv * hblocks: pairs per sequence
  int ctas;        // CTAs of the attention kernel
  int page_shift;
  float scale_log2;
  float* part_o;   // [ctas][2][kRows][head_dim]
  float* part_ml;  // [ctas][2][kRows][2]
};

__device__ __forceinline__ int keys_of(const Params& p, int seq) {
  const int64_t n = (int64_t)p.c.lens[seq] + p.c.len_add;
  return (int)min(max(n, (int64_t)0), p.c.max_pages * (int64_t)p.c.page_size);
}
__device__ __forceinline__ int first_key(const Params& p, int len) {
  return p.c.window > 0 && len > p.c.window ? len - p.c.window : 0;
}
// tiles of a sequence of `len` keys per (key head, head block)
__device__ __forceinline__ int tiles_of(const Params& p, int len) {
  return len == 0 ? 0 : (len - 1) / kTile - first_key(p, len) / kTile + 1;
}

// Position of a tile on the line of all tiles.
struct Where {
  int seq, unit, tile, ntiles;  // tile in [0, ntiles) of the pair
  int64_t first;                // the pair's first tile on the line
};

// Sum of tiles over all sequences, and where tile `at` lies. All threads of the CTA.
// `red` holds blockDim.x + 1 + blockDim.x / 32 int64.
__device__ int64_t line_total(const Params& p, int64_t* red, int per) {
  int64_t s = 0;
  for (int i = 0; i < per; ++i) {
    const int seq = threadIdx.x * per + i;
    if (seq < p.c.n_seqs) s += tiles_of(p, keys_of(p, seq));
  }
  s *= p.units;
  // inclusive scan in the warp, then over the warps
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  int64_t* wsum = red + blockDim.x + 1;
  if (lane == 31) wsum[warp] = s;
  __syncthreads();
  for (int i = 0; i < warp; ++i) s += wsum[i];
  red[threadIdx.x + 1] = s;
  if (threadIdx.x == 0) red[0] = 0;
  __syncthreads();
  return red[blockDim.x];
}

__device__ Where locate(const Params& p, const int64_t* red, int per, int64_t at) {
  // thread whose sequences hold `at`: the last prefix <= at
  int lo = 0, hi = (int)blockDim.x;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (red[mid] <= at) lo = mid;
    else hi = mid;
  }
  Where w;
  int64_t base = red[lo];
  w.seq = lo * per;
  for (;; ++w.seq) {
    w.ntiles = tiles_of(p, keys_of(p, w.seq));
    const int64_t n = (int64_t)w.ntiles * p.units;
    if (at < base + n) break;
    base += n;
  }
  const int64_t r = at - base;
  w.unit = (int)(r / w.ntiles);
  w.tile = (int)(r - (int64_t)w.unit * w.ntiles);
  w.first = at - w.tile;
  return w;
}

// shares of the line: none is empty
__device__ __forceinline__ int shares(const Params& p, int64_t total) { return (int)min((int64_t)p.ctas, total); }
__device__ __forceinline__ int64_t share_begin(int64_t total, int ctas, int64_t c) { return c * total / ctas; }
// the CTA whose share holds tile x
__device__ __forceinline__ int share_of(int64_t total, int ctas, int64_t x) {
  return (int)(((x + 1) * ctas - 1) / total);
}

// ------------------------------------------------------------------ matrix helpers
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
template <int DT>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (DT == DT_BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Row pitch 2 HD bytes; 16-byte chunk c of row r lies at chunk c ^ key(r), which puts the 8
// rows that one ldmatrix reads on distinct banks (a pitch that is an odd multiple of 64
// bytes shifts every other row by half the banks already).
template <int HD>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  const int key = (HD / 8) % 8 == 0 ? (r & 7) : ((r >> 1) & 3);
  return (uint32_t)(r * HD * 2 + ((c ^ key) << 4));
}

template <int HD>
struct Cfg {
  static constexpr int kStageWarp = 2 * 16 * HD * 2;             // K and V rows of one warp's stage
  static constexpr int kStages = HD <= 32 ? 8 : HD <= 64 ? 6 : HD <= 96 ? 4 : HD <= 192 ? 3 : 2;
  static constexpr int kCtasPerSm = HD <= 128 ? 2 : 1;
  static constexpr int kRing = kWarps * kStages * kStageWarp;
  static constexpr int kMerge = 2 * kRows * HD * 4 + 2 * kRows * 2 * 4;  // two warps' outputs and statistics
  static constexpr int kQ = HD > 128 ? kRows * HD * 2 : 0;        // wide heads read q from shared memory
  static constexpr int kSmem = kRing + kMerge + kQ;
};

template <int HD, int DT>
__global__ void __launch_bounds__(kThreads, Cfg<HD>::kCtasPerSm) attention_kernel(const __grid_constant__ Params p) {
  using C = Cfg<HD>;
  constexpr int ST = C::kStages, KS = HD / 16, CH = HD / 8;
  extern __shared__ __align__(128) uint8_t smem[];
  int64_t* red = reinterpret_cast<int64_t*>(smem + C::kRing);  // before the merge boxes are in use
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const AttnCall& c = p.c;
  grid_wait();

  const int per = (c.n_seqs + kThreads - 1) / kThreads;
  const int64_t total = line_total(p, red, per);
  // sequences without keys: their rows are zero (split over the CTAs)
  for (int s = blockIdx.x; s < c.n_seqs; s += gridDim.x) {
    if ((int64_t)c.lens[s] + c.len_add > c.max_pages * c.page_size) report(c.status, 6 /* HARP_ERR_DEVICE_CHECK */, 93);
    if ((c.keep_negative && c.lens[s] < 0) || keys_of(p, s) != 0) continue;  // a negative length leaves the row as it was
    for (int i = threadIdx.x; i < c.n_heads * HD; i += kThreads)
      store_act(c.out, s * c.o_ss + (i / HD) * c.o_hs + i % HD, DT, 0.f);
    if (c.lse)
      for (int i = threadIdx.x; i < c.n_heads; i += kThreads) c.lse[(int64_t)s * c.n_heads + i] = -INFINITY;
  }
  const int ctas = shares(p, total);
  if ((int)blockIdx.x >= ctas) {
    grid_release();
    return;
  }
  const int64_t begin = share_begin(total, ctas, blockIdx.x), end = share_begin(total, ctas, blockIdx.x + 1);

  const uint32_t ring = smem_u32(smem) + warp * ST * C::kStageWarp;
  float* merge_o = reinterpret_cast<float*>(smem + C::kRing);        // [2][kRows][HD]
  float* merge_ml = merge_o + 2 * kRows * HD;                        // [2][kRows][2]
  const uint32_t q_s = smem_u32(smem + C::kRing + C::kMerge);

  // ---------------- load cursor: runs ST - 1 tiles ahead of the products
  const Where w0 = locate(p, red, per, begin);
  Where lw = w0;
  int64_t l_at = begin;
  int l_len = keys_of(p, lw.seq), l_start = first_key(p, l_len);
  // lane j < 16 holds the page of the warp's key j of the tile the cursor stands on
  auto page_ahead = [&]() -> int {
    const int key = (l_start / kTile + lw.tile) * kTile + warp * 16 + (lane & 15);
    return key >= l_start && key < l_len ? c.table[(int64_t)lw.seq * c.table_stride + (key >> p.page_shift)] : -1;
  };
  int page = page_ahead();
  auto load_tile = [&](int slot) {
    const uint32_t dst = ring + slot * C::kStageWarp;
    const int key = (l_start / kTile + lw.tile) * kTile + warp * 16 + (lane & 15);
    int64_t off = -1;
    if (key >= l_start && key < l_len) {
      if (page >= 0 && page < c.n_pages)
        off = page * c.page_stride + (int64_t)(key & (c.page_size - 1)) * c.row_stride +
              (int64_t)(lw.unit / p.hblocks) * c.head_stride;
      else report(c.status, 6 /* HARP_ERR_DEVICE_CHECK */, 92);  // a row that is not there reads as zeros
    }
#pragma unroll
    for (int i = 0; i < CH * 16 / 32; ++i) {
      const int x = i * 32 + lane, r = x / CH, ch = x % CH;
      const int64_t ro = __shfl_sync(0xffffffffu, off, r);
      const int64_t eo = (ro < 0 ? 0 : ro) + ch * 8;
      const uint32_t at = chunk_at<HD>(r, ch);
      cp_async16(dst + at, static_cast<const uint16_t*>(c.kc) + eo, ro >= 0);
      cp_async16(dst + 16 * HD * 2 + at, static_cast<const uint16_t*>(c.vc) + eo, ro >= 0);
    }
    // advance, and ask for the next tile's pages
    ++l_at;
    if (l_at < end) {
      if (++lw.tile == lw.ntiles) {
        lw.tile = 0;
        if (++lw.unit == p.units) {
          lw.unit = 0;
          do {
            ++lw.seq;
            l_len = keys_of(p, lw.seq);
            lw.ntiles = tiles_of(p, l_len);
          } while (lw.ntiles == 0);
          l_start = first_key(p, l_len);
        }
      }
      page = page_ahead();
    }
  };

  int put = 0;
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) {
    if (l_at < end) load_tile(put++);
    cp_commit();
  }

  // ---------------- products
  Where w = w0;
  int len = keys_of(p, w.seq), start = first_key(p, len);
  int64_t at = begin;
  int slot = 0;
  while (at < end) {
    const int kvh = w.unit / p.hblocks, hb = w.unit - kvh * p.hblocks;
    const int h0 = kvh * p.group + hb * kRows, nh = min(kRows, p.group - hb * kRows);
    const int tile_end = (int)min((int64_t)w.ntiles, w.tile + (end - at));
    const int row = lane >> 2;
    // q rows `row` and `row + 8` as A fragments (rows beyond the group are zero)
    uint32_t qf[HD > 128 ? 1 : KS][4];
    {
      const uint16_t* q = static_cast<const uint16_t*>(c.q) + w.seq * c.q_ss + h0 * c.q_hs;
      auto pair_at = [&](int r, int d) -> uint32_t {
        if (r >= nh) return 0u;
        return *reinterpret_cast<const uint32_t*>(q + r * c.q_hs + d);
      };
      if (HD > 128) {
        __syncthreads();  // the last pair's q is no longer read
        for (int i = threadIdx.x; i < kRows * HD / 2; i += kThreads) {
          const int r = i / (HD / 2), d = (i % (HD / 2)) * 2;
          *reinterpret_cast<uint32_t*>(smem + C::kRing + C::kMerge + chunk_at<HD>(r, d >> 3) + (d & 7) * 2) = pair_at(r, d);
        }
        __syncthreads();
      } else {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int d = k * 16 + (lane & 3) * 2;
          qf[HD > 128 ? 0 : k][0] = pair_at(row, d);
          qf[HD > 128 ? 0 : k][1] = pair_at(row + 8, d);
          qf[HD > 128 ? 0 : k][2] = pair_at(row, d + 8);
          qf[HD > 128 ? 0 : k][3] = pair_at(row + 8, d + 8);
        }
      }
    }
    float o[HD / 8][4];
#pragma unroll
    for (int i = 0; i < HD / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    for (int tile = w.tile; tile < tile_end; ++tile) {
      cp_wait<ST - 2>();
      __syncwarp();
      // the stage refilled here was read before this __syncwarp
      if (l_at < end) {
        load_tile(put);
        put = put + 1 == ST ? 0 : put + 1;
      }
      cp_commit();
      const uint32_t ks = ring + slot * C::kStageWarp, vs = ks + 16 * HD * 2;
      // scores of 16 keys: two blocks of 8
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t b[4];
        ldsm4(b, ks + chunk_at<HD>((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
        if (HD > 128) {
          uint32_t a[4];
          ldsm4(a, q_s + chunk_at<HD>(lane & 15, 2 * k + (lane >> 4)));
          mma16816<DT>(s[0], a, b[0], b[1]);
          mma16816<DT>(s[1], a, b[2], b[3]);
        } else {
          mma16816<DT>(s[0], qf[HD > 128 ? 0 : k], b[0], b[1]);
          mma16816<DT>(s[1], qf[HD > 128 ? 0 : k], b[2], b[3]);
        }
      }
      const int key0 = (start / kTile + tile) * kTile + warp * 16 + (lane & 3) * 2;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = key0 + j * 8 + (e & 1);
          s[j][e] = key >= start && key < len ? s[j][e] * p.scale_log2 : -INFINITY;
        }
      float n0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
      float n1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
#pragma unroll
      for (int x = 1; x < 4; x <<= 1) {
        n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, x));
        n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, x));
      }
      n0 = fmaxf(m0, n0);
      n1 = fmaxf(m1, n1);
      if (__any_sync(0xffffffffu, n0 > m0 || n1 > m1)) {
        // -inf: no live key yet, nothing to rescale
        const float f0 = m0 == -INFINITY ? 0.f : exp2f(m0 - n0), f1 = m1 == -INFINITY ? 0.f : exp2f(m1 - n1);
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) {
          o[i][0] *= f0;
          o[i][1] *= f0;
          o[i][2] *= f1;
          o[i][3] *= f1;
        }
        m0 = n0;
        m1 = n1;
      }
      const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float a = exp2f(s[j][0] - z0), b = exp2f(s[j][1] - z0), d = exp2f(s[j][2] - z1), e = exp2f(s[j][3] - z1);
        l0 += a + b;
        l1 += d + e;
        hi[2 * j] = pack2(a, b, DT);
        hi[2 * j + 1] = pack2(d, e, DT);
        const float2 x = unpack2(hi[2 * j], DT), y = unpack2(hi[2 * j + 1], DT);
        lo[2 * j] = pack2(a - x.x, b - x.y, DT);
        lo[2 * j + 1] = pack2(d - y.x, e - y.y, DT);
      }
#pragma unroll
      for (int i = 0; i < HD / 16; ++i) {
        uint32_t b[4];
        ldsm4t(b, vs + chunk_at<HD>((lane & 7) + (((lane >> 3) & 1) << 3), 2 * i + (lane >> 4)));
        mma16816<DT>(o[2 * i], hi, b[0], b[1]);
        mma16816<DT>(o[2 * i + 1], hi, b[2], b[3]);
        mma16816<DT>(o[2 * i], lo, b[0], b[1]);
        mma16816<DT>(o[2 * i + 1], lo, b[2], b[3]);
      }
      slot = slot + 1 == ST ? 0 : slot + 1;
    }

    // ---------------- join the four warps (1 -> 0 and 3 -> 2, then 2 -> 0), in key order
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, x);
      l1 += __shfl_xor_sync(0xffffffffu, l1, x);
    }
#pragma unroll
    for (int step = 1; step <= 2; ++step) {
      const bool gives = step == 1 ? (warp & 1) : warp == 2, takes = step == 1 ? !(warp & 1) : warp == 0;
      const int box = step == 1 ? warp >> 1 : 0;
      float* bo = merge_o + box * kRows * HD;
      float* bml = merge_ml + box * kRows * 2;
      __syncthreads();  // the boxes are free
      if (gives) {
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) {
          const int d = i * 8 + (lane & 3) * 2;
          *reinterpret_cast<float2*>(bo + row * HD + d) = make_float2(o[i][0], o[i][1]);
          *reinterpret_cast<float2*>(bo + (row + 8) * HD + d) = make_float2(o[i][2], o[i][3]);
        }
        if ((lane & 3) == 0) {
          bml[row * 2] = m0;
          bml[row * 2 + 1] = l0;
          bml[(row + 8) * 2] = m1;
          bml[(row + 8) * 2 + 1] = l1;
        }
      }
      __syncthreads();
      if (takes) {
        const float a0 = bml[row * 2], a1 = bml[(row + 8) * 2];
        const float n0 = fmaxf(m0, a0), n1 = fmaxf(m1, a1);
        const float f0 = m0 == -INFINITY ? 0.f : exp2f(m0 - n0), f1 = m1 == -INFINITY ? 0.f : exp2f(m1 - n1);
        const float g0 = a0 == -INFINITY ? 0.f : exp2f(a0 - n0), g1 = a1 == -INFINITY ? 0.f : exp2f(a1 - n1);
        l0 = l0 * f0 + bml[row * 2 + 1] * g0;
        l1 = l1 * f1 + bml[(row + 8) * 2 + 1] * g1;
        m0 = n0;
        m1 = n1;
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) {
          const int d = i * 8 + (lane & 3) * 2;
          const float2 x = *reinterpret_cast<const float2*>(bo + row * HD + d);
          const float2 y = *reinterpret_cast<const float2*>(bo + (row + 8) * HD + d);
          o[i][0] = o[i][0] * f0 + x.x * g0;
          o[i][1] = o[i][1] * f0 + x.y * g0;
          o[i][2] = o[i][2] * f1 + y.x * g1;
          o[i][3] = o[i][3] * f1 + y.y * g1;
        }
      }
    }

    // ---------------- the pair's output, or this share's partial of it
    if (warp == 0) {
      const bool whole = w.tile == 0 && tile_end == w.ntiles;
      if (whole) {
        const float i0 = 1.f / l0, i1 = 1.f / l1;
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) {
          const int d = i * 8 + (lane & 3) * 2;
          uint16_t* out = static_cast<uint16_t*>(c.out) + w.seq * c.o_ss + h0 * c.o_hs + d;
          if (row < nh) *reinterpret_cast<uint32_t*>(out + row * c.o_hs) = pack2(o[i][0] * i0, o[i][1] * i0, DT);
          if (row + 8 < nh) *reinterpret_cast<uint32_t*>(out + (row + 8) * c.o_hs) = pack2(o[i][2] * i1, o[i][3] * i1, DT);
        }
        if (c.lse && (lane & 3) == 0) {
          float* lse = c.lse + (int64_t)w.seq * c.n_heads + h0;
          if (row < nh) lse[row] = (m0 + log2f(l0)) * 0.69314718055994530942f;
          if (row + 8 < nh) lse[row + 8] = (m1 + log2f(l1)) * 0.69314718055994530942f;
        }
      } else {
        const int64_t box = (int64_t)blockIdx.x * 2 + (at == begin ? 0 : 1);
        float* po = p.part_o + box * kRows * HD;
        float* pml = p.part_ml + box * kRows * 2;
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) {
          const int d = i * 8 + (lane & 3) * 2;
          *reinterpret_cast<float2*>(po + row * HD + d) = make_float2(o[i][0], o[i][1]);
          *reinterpret_cast<float2*>(po + (row + 8) * HD + d) = make_float2(o[i][2], o[i][3]);
        }
        if ((lane & 3) == 0) {
          pml[row * 2] = m0;
          pml[row * 2 + 1] = l0;
          pml[(row + 8) * 2] = m1;
          pml[(row + 8) * 2 + 1] = l1;
        }
      }
    }
    // ---------------- next pair
    at += tile_end - w.tile;
    if (at < end) {
      w.tile = 0;
      if (++w.unit == p.units) {
        w.unit = 0;
        do {
          ++w.seq;
          len = keys_of(p, w.seq);
          w.ntiles = tiles_of(p, len);
        } while (w.ntiles == 0);
        start = first_key(p, len);
      }
    }
  }
  cp_wait<0>();
  grid_release();
}

// Joins the partials of the pairs that a share border cuts. CTA (b, g): the pair cut by the
// border in front of share b, if that is the pair's first cut; heads kJoinRows * g onward.
template <int HD, int DT>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Params p) {
  __shared__ int64_t red[kJoinThreads + 1 + kJoinThreads / 32];
  const AttnCall& c = p.c;
  grid_wait();
  const int per = (c.n_seqs + kJoinThreads - 1) / kJoinThreads;
  const int64_t total = line_total(p, red, per);
  const int b = blockIdx.x + 1;
  const int ctas = shares(p, total);
  if (b >= ctas) return;
  const int64_t border = share_begin(total, ctas, b);
  const Where w = locate(p, red, per, border);
  const int64_t a = w.first, e = a + w.ntiles;
  if (border == a) return;                             // the border lies between two pairs
  const int c0 = share_of(total, ctas, a), c1 = share_of(total, ctas, e - 1);
  if (b != c0 + 1) return;                             // not the pair's first cut
  const int kvh = w.unit / p.hblocks, hb = w.unit - kvh * p.hblocks;
  const int h0 = kvh * p.group + hb * kRows, nh = min(kRows, p.group - hb * kRows);
  const int r0 = blockIdx.y * kJoinRows;
  const bool first_is_second = share_begin(total, ctas, c0) < a;  // share c0 began before the pair
  for (int i = threadIdx.x; i < kJoinRows * (HD / 4); i += kJoinThreads) {
    const int r = r0 + i / (HD / 4), d = (i % (HD / 4)) * 4;
    if (r >= nh) break;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int x = c0; x <= c1; ++x) {
      const int64_t box = (int64_t)x * 2 + (x == c0 && first_is_second ? 1 : 0);
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + (box * kRows + r) * 2);
      const float4 v = *reinterpret_cast<const float4*>(p.part_o + (box * kRows + r) * HD + d);
      const float n = fmaxf(m, ml.x);
      const float f = m == -INFINITY ? 0.f : exp2f(m - n), g = ml.x == -INFINITY ? 0.f : exp2f(ml.x - n);
      m = n;
      l = l * f + ml.y * g;
      o.x = o.x * f + v.x * g;
      o.y = o.y * f + v.y * g;
      o.z = o.z * f + v.z * g;
      o.w = o.w * f + v.w * g;
    }
    const float inv = 1.f / l;
    uint16_t* out = static_cast<uint16_t*>(c.out) + w.seq * c.o_ss + (h0 + r) * c.o_hs + d;
    reinterpret_cast<uint32_t*>(out)[0] = pack2(o.x * inv, o.y * inv, DT);
    reinterpret_cast<uint32_t*>(out)[1] = pack2(o.z * inv, o.w * inv, DT);
    if (c.lse && d == 0) c.lse[(int64_t)w.seq * c.n_heads + h0 + r] = (m + log2f(l)) * 0.69314718055994530942f;
  }
}

template <int HD, int DT>
cudaError_t launch_t(Params& p, cudaStream_t st) {
  using C = Cfg<HD>;
  int dev = 0;
  cudaGetDevice(&dev);
  static bool attr_done[64] = {false};  // per device
  if (dev < 0 || dev >= 64 || !attr_done[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(attention_kernel<HD, DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_done[dev] = true;
  }
  p.ctas = 148 * C::kCtasPerSm;
  p.part_o = static_cast<float*>(p.c.ws);
  p.part_ml = p.part_o + (int64_t)p.ctas * 2 * kRows * HD;
  cudaError_t e = launch_dependent(attention_kernel<HD, DT>, dim3(p.ctas), dim3(kThreads), C::kSmem, st, p);
  if (e != cudaSuccess) return e;
  const int groups = (min(p.group, kRows) + kJoinRows - 1) / kJoinRows;
  return launch_dependent(join_kernel<HD, DT>, dim3(p.ctas - 1, groups), dim3(kJoinThreads), 0, st, p);
}

template <int DT>
cudaError_t launch_dt(Params& p, cudaStream_t st) {
  switch (p.c.head_dim) {
    case 32: return launch_t<32, DT>(p, st);
    case 64: return launch_t<64, DT>(p, st);
    case 96: return launch_t<96, DT>(p, st);
    case 128: return launch_t<128, DT>(p, st);
    case 192: return launch_t<192, DT>(p, st);
    case 256: return launch_t<256, DT>(p, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

size_t attention_ws_bytes(int head_dim) { return (size_t)kMaxCtas * 2 * kRows * (head_dim + 2) * sizeof(float); }

const char* attention_refuses(int n_seqs, int n_heads, int n_kv, int head_dim, int dt) {
  if (n_seqs < 0 || n_seqs > 65535 || n_heads < 1 || n_heads > 65535 || n_kv < 1 || n_heads % n_kv) return "bad sizes";
  if (dt != DT_BF16 && dt != DT_F16) return "bf16 or f16 only";
  for (int d : {32, 64, 96, 128, 192, 256})
    if (head_dim == d) return nullptr;
  return "head_dim must be 32, 64, 96, 128, 192 or 256";
}

cudaError_t launch_attention(const AttnCall& c, cudaStream_t st) {
  Params p{};
  p.c = c;
  p.group = c.n_heads / c.n_kv;
  p.hblocks = (p.group + kRows - 1) / kRows;
  p.units = c.n_kv * p.hblocks;
  while ((1 << p.page_shift) < c.page_size) ++p.page_shift;
  p.scale_log2 = c.scale * 1.44269504088896340736f;
  return c.dt == DT_BF16 ? launch_dt<DT_BF16>(p, st) : launch_dt<DT_F16>(p, st);
}

}  // namespace harp

using namespace harp;

extern "C" {

harp_status harp_paged_attention_workspace_size(int head_dim, size_t* bytes) {
  if (!bytes || head_dim < 1 || head_dim > 256) return set_error(HARP_ERR_INVALID_ARG, "paged_attention_workspace_size: bad arguments");
  *bytes = attention_ws_bytes(head_dim);
  return HARP_OK;
}

harp_status harp_paged_attention(const harp_kv_cache* cache, int n_seqs, int n_heads, const void* q, int64_t q_seq_stride,
                                 int64_t q_head_stride, const int32_t* page_table, int64_t max_pages, const int32_t* seq_lens,
                                 float scale, int window, void* out, int64_t o_seq_stride, int64_t o_head_stride, float* lse,
                                 void* workspace, size_t ws_bytes, void* stream) {
  harp_status s = check_cache("paged_attention", cache);
  if (s != HARP_OK) return s;
  if (!q || !page_table || !seq_lens || !out) return set_error(HARP_ERR_INVALID_ARG, "paged_attention: null pointer");
  if (const char* why = attention_refuses(n_seqs, n_heads, cache->n_kv_heads, cache->head_dim, cache->dtype))
    return set_error(why[0] == 'h' ? HARP_ERR_UNSUPPORTED : HARP_ERR_INVALID_ARG, "paged_attention: %s", why);
  if (max_pages < 1 || max_pages * cache->page_size > 0x7fffff00) return set_error(HARP_ERR_INVALID_ARG, "paged_attention: max_pages out of range");
  if (window < 0 || !(scale == scale)) return set_error(HARP_ERR_INVALID_ARG, "paged_attention: bad scale or window");
  if (!aligned_to(q, 4) || !aligned_to(out, 4) || (q_seq_stride | q_head_stride | o_seq_stride | o_head_stride) & 1)
    return set_error(HARP_ERR_INVALID_ARG, "paged_attention: rows of q and out must lie on 4-byte boundaries");
  if (!aligned_to(page_table, 4) || !aligned_to(seq_lens, 4) || !aligned_to(lse, 4))
    return set_error(HARP_ERR_INVALID_ARG, "paged_attention: a pointer is not aligned to its type");
  if (!workspace || ws_bytes < attention_ws_bytes(cache->head_dim) || !aligned_to(workspace, 256))
    return set_error(HARP_ERR_WORKSPACE, "paged_attention: workspace of %zu bytes (256-byte aligned) needed", attention_ws_bytes(cache->head_dim));
  if (n_seqs == 0) return HARP_OK;
  AttnCall c{};
  if ((s = device_status_for_kernels(&c.status)) != HARP_OK) return s;
  c.n_seqs = n_seqs;
  c.n_heads = n_heads;
  c.n_kv = cache->n_kv_heads;
  c.head_dim = cache->head_dim;
  c.dt = cache->dtype;
  c.q = q;
  c.q_ss = q_seq_stride;
  c.q_hs = q_head_stride;
  c.kc = cache->k;
  c.vc = cache->v;
  c.page_size = cache->page_size;
  c.n_pages = cache->n_pages;
  c.page_stride = cache->page_stride;
  c.head_stride = cache->head_stride;
  c.row_stride = cache->row_stride;
  c.max_pages = max_pages;
  c.table = page_table;
  c.table_stride = max_pages;
  c.lens = seq_lens;
  c.keep_negative = 1;
  c.scale = scale;
  c.window = window;
  c.out = out;
  c.o_ss = o_seq_stride;
  c.o_hs = o_head_stride;
  c.lse = lse;
  c.ws = workspace;
  const cudaError_t e = launch_attention(c, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HARP_OK : set_error(HARP_ERR_CUDA, "paged_attention launch: %s", cudaGetErrorString(e));
}

}  // extern "C"
