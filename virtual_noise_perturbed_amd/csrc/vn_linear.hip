// Linear layer with its epilogue, and its gradients (gfx950):
//   z = x W^T + b,   y = act(z) + residual
//   dz = dy act'(z), dx = dz W,  dW = dz^T x,  db = sum over rows of dz
// Every product is one form, C[m,n] = sum_k A[m,k] B[n,k], with both operands
// contiguous along k, on the bf16 matrix cores with fp32 accumulation:
//   - bf16 operands as they are;
//   - fp32 operands as three bf16 values each, v = h + m + l (h = bf16(v),
//     m = bf16(v - h), l = bf16(v - h - m): 24 bits and more), and the six
//     products hh, hm, mh, hl, mm, lh; what is dropped is below 2^-24 of a
//     product.  Six bf16 products at 16x the fp32 matrix rate take 0.4 of the
//     fp32 matrix cores' time.
// pack_kernel brings an operand into this form where it is not: transposed
// (W for dx; dz and x for dW), in three planes, padded along k to whole stages
// of 64, or multiplied by act'(z).  dz is rounded to bf16 for the products of
// bf16 operands; db is summed from the unrounded dz.
#include <stdint.h>

#include <utility>

#include "vn_dense.hpp"
#include "vn_rows.hpp"

namespace vn {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int BK = 64;   // k per stage

// ---- activations -----------------------------------------------------------

__device__ __forceinline__ float act_value(Act a, float z) {
  switch (a) {
    case Act::relu: return z > 0.0f ? z : 0.0f;
    case Act::gelu: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    case Act::silu: return z / (1.0f + expf(-z));
    case Act::gelu_tanh: {
      // (1 + tanh u) / 2 = 1 / (1 + exp(-2u))
      const float u = 0.79788456080286536f * (z + 0.044715f * z * z * z);
      return z / (1.0f + expf(-2.0f * u));
    }
    default: return z;
  }
}

__device__ __forceinline__ float act_slope(Act a, float z) {
  switch (a) {
    case Act::relu: return z > 0.0f ? 1.0f : 0.0f;
    case Act::gelu:
      return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) + z * expf(-0.5f * z * z) * 0.39894228040143268f;
    case Act::silu: {
      const float s = 1.0f / (1.0f + expf(-z));
      return s * (1.0f + z * (1.0f - s));
    }
    case Act::gelu_tanh: {
      const float u = 0.79788456080286536f * (z + 0.044715f * z * z * z);
      const float s = 1.0f / (1.0f + expf(-2.0f * u));
      const float du = 0.79788456080286536f * (1.0f + 3.0f * 0.044715f * z * z);
      return s + z * s * (1.0f - s) * 2.0f * du;
    }
    default: return 1.0f;
  }
}

// ---- epilogue --------------------------------------------------------------

struct Epilogue {
  const float* bias;     // by column, or null
  const void* residual;  // in out_type, or null
  Act act;
  Elem out_type, pre_type;
  void* out;             // (m, n) dense
  void* pre;             // or null
};

__device__ __forceinline__ float load_elem(const void* p, Elem t, int64_t i) {
  return t == Elem::f32 ? static_cast<const float*>(p)[i] : static_cast<float>(static_cast<const __bf16*>(p)[i]);
}
__device__ __forceinline__ void store_elem(void* p, Elem t, int64_t i, float v) {
  if (t == Elem::f32) static_cast<float*>(p)[i] = v;
  else static_cast<__bf16*>(p)[i] = static_cast<__bf16>(v);
}

// Output i (column's bias b) from the product's value.
__device__ __forceinline__ void finish(const Epilogue& e, int64_t i, float b, float acc) {
  const float z = acc + b;
  if (e.pre != nullptr) store_elem(e.pre, e.pre_type, i, z);
  float y = act_value(e.act, z);
  if (e.residual != nullptr) y += load_elem(e.residual, e.out_type, i);
  store_elem(e.out, e.out_type, i, y);
}

// ---- the product -----------------------------------------------------------

struct Product {
  const __bf16* a;       // (m, lda), planes a_plane apart
  const __bf16* b;       // (n, ldb), planes b_plane apart
  int64_t a_plane, b_plane, lda, ldb;
  int64_t m, n;
  int32_t nk;            // stages of BK along k
  int32_t terms;         // 1, or 6 for three planes
  int32_t tiles_m, tiles_n, splits;
  float* partial;        // (splits, m, n) when splits > 1
  Epilogue e;
};

// Planes (0 h, 1 m, 2 l) of the six products of fp32 operands, smallest first;
// two bits each.
constexpr uint32_t kPlanesA = 2u << 0 | 1u << 2 | 0u << 4 | 1u << 6 | 0u << 8 | 0u << 10;
constexpr uint32_t kPlanesB = 0u << 0 | 1u << 2 | 2u << 4 | 0u << 6 | 1u << 8 | 0u << 10;

// LDS layout of a stage: unit (16 B) of (row r, k-segment s of 8) is
// r*8 + (s ^ swz(r)); the swizzle keeps the fragment reads (32 rows at one
// segment) free of bank conflicts.
__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// 16 bytes at each lane's address -> LDS byte address base + IMM + 16 * lane
// (base wave-uniform).  M0 takes the LDS address; one wait state separates its
// write from the load.  Nothing tracks the load: wait_vm before its use.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int IMM>
__device__ __forceinline__ void lds_load16(const void* p, uint32_t base) {
  asm volatile("s_add_u32 m0, %1, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "s"(base), "n"(IMM)
               : "memory", "m0", "scc");
}
#pragma clang diagnostic pop
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <typename F, int... I>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_impl(f, std::make_integer_sequence<int, N>{});
}

// Tile q of a tiles_m x tiles_n grid for workgroup `id`: consecutive ids go to
// the 8 XCDs in turn; each XCD takes a contiguous range of an order that walks
// groups of 4 row tiles column by column, so that its tiles share rows of A
// and B in its L2.
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm, uint32_t& tn) {
  const uint32_t total = tiles_m * tiles_n;
  const uint32_t x = id % 8, i = id / 8, per = total / 8, rest = total % 8;
  const uint32_t q = x * per + (x < rest ? x : rest) + i;
  const uint32_t first = q / (4 * tiles_n) * 4;
  const uint32_t gsz = (tiles_m - first) < 4 ? (tiles_m - first) : 4;
  const uint32_t r = q - first * tiles_n;
  tm = first + r % gsz;
  tn = r / gsz;
}

// One tile of TM x TN outputs by 4 waves (2 x 2), two LDS slots of a stage:
// stage s + 1 is on its way while stage s is multiplied.  Rows past m or n are
// read from the last row and not stored.
template <int TM, int TN>
__global__ __launch_bounds__(256, 2) void tile_kernel(Product g) {
  constexpr int UNITS = (TM + TN) * 8, LOADS = UNITS / 256;
  constexpr int MB = TM / 64, NB = TN / 64;   // 32-blocks per wave
  __shared__ uint4 smem[2 * UNITS];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  uint32_t tm, tn;
  tile_of(blockIdx.x, g.tiles_m, g.tiles_n, tm, tn);
  const int64_t m0 = static_cast<int64_t>(tm) * TM, n0 = static_cast<int64_t>(tn) * TN;

  const int lrow = tid >> 3;
  const int lseg = (tid & 7) ^ swz(lrow);
  const uint32_t wave_lds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(smem)) + wave * 64 * 16;
  const __bf16* src[LOADS];
#pragma unroll
  for (int u = 0; u < LOADS; ++u) {
    const int row = u * 32 + lrow;
    if (u * 32 < TM) {
      const int64_t r = m0 + row < g.m ? m0 + row : g.m - 1;
      src[u] = g.a + r * g.lda + lseg * 8;
    } else {
      const int64_t r = n0 + (row - TM) < g.n ? n0 + (row - TM) : g.n - 1;
      src[u] = g.b + r * g.ldb + lseg * 8;
    }
  }
  const int stages = g.nk * g.terms;
  const int per = (stages + g.splits - 1) / g.splits;
  const int begin = static_cast<int>(blockIdx.y) * per;
  const int end = begin + per < stages ? begin + per : stages;
  auto load_stage = [&](int s, int slot) {
    const int term = s / g.nk;
    const int64_t k = static_cast<int64_t>(s - term * g.nk) * BK;
    const int64_t ka = k + ((g.terms > 1 ? (kPlanesA >> (2 * term)) & 3 : 0) * g.a_plane);
    const int64_t kb = k + ((g.terms > 1 ? (kPlanesB >> (2 * term)) & 3 : 0) * g.b_plane);
    const uint32_t base = __builtin_amdgcn_readfirstlane(wave_lds + slot * (UNITS * 16));
    static_for<LOADS>([&](auto uc) {
      constexpr int u = decltype(uc)::value;
      lds_load16<u * 256 * 16>(src[u] + (u * 32 < TM ? ka : kb), base);
    });
  };

  const int l32 = lane & 31, lh = lane >> 5;
  const int swl = swz(l32);
  const int arow = (wm * (TM / 2) + l32) * 8;
  const int brow = TM * 8 + (wn * (TN / 2) + l32) * 8;
  f32x16 acc[MB][NB];
#pragma unroll
  for (int a = 0; a < MB; ++a)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[a][b] = f32x16{};

  if (begin < end) load_stage(begin, 0);
  for (int s = begin; s < end; ++s) {
    const int slot = (s - begin) & 1;
    wait_vm<0>();
    __syncthreads();   // stage s is whole; the other slot's readers are done
    if (s + 1 < end) load_stage(s + 1, slot ^ 1);
    const uint4* st = smem + slot * UNITS;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int seg = (2 * t + lh) ^ swl;
      bf16x8 fa[MB], fb[NB];
#pragma unroll
      for (int a = 0; a < MB; ++a) fa[a] = __builtin_bit_cast(bf16x8, st[arow + a * 256 + seg]);
#pragma unroll
      for (int b = 0; b < NB; ++b) fb[b] = __builtin_bit_cast(bf16x8, st[brow + b * 256 + seg]);
#pragma unroll
      for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[a], fb[b], acc[a][b], 0, 0, 0);
    }
  }

  // Lane l holds column l % 32 of each 32-block and rows
  // 8 * (v / 4) + 4 * (l / 32) + v % 4 for v < 16.
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int64_t n = n0 + wn * (TN / 2) + b * 32 + l32;
    if (n >= g.n) continue;
    const float bias = g.e.bias != nullptr && g.splits == 1 ? g.e.bias[n] : 0.0f;
#pragma unroll
    for (int a = 0; a < MB; ++a) {
      const int64_t mb = m0 + wm * (TM / 2) + a * 32 + 4 * lh;
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int64_t m = mb + 8 * (v >> 2) + (v & 3);
        if (m >= g.m) continue;
        if (g.splits > 1) g.partial[(static_cast<int64_t>(blockIdx.y) * g.m + m) * g.n + n] = acc[a][b][v];
        else finish(g.e, m * g.n + n, bias, acc[a][b][v]);
      }
    }
  }
}

// Joins the splits' partial products in split order and finishes them.
__global__ __launch_bounds__(256) void join_kernel(Product g) {
  const int64_t total = g.m * g.n;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    float t = 0.0f;
    for (int s = 0; s < g.splits; ++s) t += g.partial[s * total + i];
    finish(g.e, i, g.e.bias != nullptr ? g.e.bias[i % g.n] : 0.0f, t);
  }
}

// ---- packing ---------------------------------------------------------------

struct Pack {
  const void* src;       // (r, c)
  Elem type;
  const void* pre;       // dz = src * act'(pre), or null
  Elem pre_type;
  Act act;
  int64_t r, c;
  int32_t planes;        // 1 or 3
  __bf16* rows;          // (r, ceil64(c)), planes rows_plane apart, or null
  int64_t rows_plane;
  __bf16* cols;          // (c, ceil64(r)), the transpose, or null
  int64_t cols_plane;
  float* sums;           // (ceil(r / 64), c): sums of 64 rows, or null
};

__device__ __forceinline__ Run8<float> load_any(const void* p, Elem t, int64_t row, int64_t c, int64_t n) {
  float v[8];
  if (t == Elem::f32) run_values(load_run(static_cast<const float*>(p) + row * n, c, n), v);
  else run_values(load_run(static_cast<const __bf16*>(p) + row * n, c, n), v);
  return make_run(v, static_cast<const float*>(nullptr));
}

// The next plane of v and what it leaves: bf16(v), nearest even (towards zero
// where that would overflow), and v minus it.
__device__ __forceinline__ float next_plane(float& v) {
  float h = static_cast<float>(static_cast<__bf16>(v));
  if (fabsf(h) == __builtin_inff() && fabsf(v) < __builtin_inff())
    h = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) & 0xFFFF0000u);
  v -= h;
  return h;
}

// 64 x 64 elements per workgroup: each thread takes 8 columns of two rows.
// The transpose goes through LDS as dwords of a column's two rows.
__global__ __launch_bounds__(256) void pack_kernel(Pack p) {
  constexpr int PITCH = 33;   // dwords per column: writes of a wave hit 64 banks
  __shared__ uint32_t tile[64 * PITCH];
  __shared__ float colsum[4 * 64];
  const int64_t ct = (p.c + 63) / 64, rt = (p.r + 63) / 64;
  const int64_t cp = ct * 64, rp = rt * 64;
  const int tid = threadIdx.x, seg = tid & 7, pair = tid >> 3;
  for (int64_t id = blockIdx.x; id < ct * rt; id += gridDim.x) {
    const int64_t r0 = id / ct * 64, c0 = id % ct * 64;
    const int64_t c = c0 + seg * 8;
    float v[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t r = r0 + 2 * pair + h;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[h][i] = 0.0f;
      if (r < p.r) {
        run_values(load_any(p.src, p.type, r, c, p.c), v[h]);
        if (p.pre != nullptr) {
          float z[8];
          run_values(load_any(p.pre, p.pre_type, r, c, p.c), z);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[h][i] *= act_slope(p.act, z[i]);
        }
      }
    }
    if (p.sums != nullptr) {
      // a wave holds 8 pairs of rows: over its lanes of one segment, then over the waves
      float s[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[i] = v[0][i] + v[1][i];
#pragma unroll
        for (int o = 8; o < 64; o *= 2) s[i] += __shfl_xor(s[i], o, 64);
      }
      if ((tid & 63) < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) colsum[(tid >> 6) * 64 + seg * 8 + i] = s[i];
      }
      __syncthreads();
      if (tid < 64 && c0 + tid < p.c)
        p.sums[id / ct * p.c + c0 + tid] = ((colsum[tid] + colsum[64 + tid]) + colsum[128 + tid]) + colsum[192 + tid];
      __syncthreads();
    }
    for (int q = 0; q < p.planes; ++q) {
      uint32_t w[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = next_plane(v[h][2 * i]), b = next_plane(v[h][2 * i + 1]);
          w[h][i] = pack_bf16(a, b);
        }
      if (p.rows != nullptr) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t r = r0 + 2 * pair + h;
          if (r < p.r) *reinterpret_cast<uint4*>(p.rows + q * p.rows_plane + r * cp + c) = make_uint4(w[h][0], w[h][1], w[h][2], w[h][3]);
        }
      }
      if (p.cols != nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          tile[(seg * 8 + 2 * i) * PITCH + pair] = (w[0][i] & 0xFFFFu) | (w[1][i] << 16);
          tile[(seg * 8 + 2 * i + 1) * PITCH + pair] = (w[0][i] >> 16) | (w[1][i] & 0xFFFF0000u);
        }
        __syncthreads();
        const int col = tid >> 2, part = tid & 3;   // 16 rows of a column
        if (c0 + col < p.c) {
          uint32_t t[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) t[i] = tile[col * PITCH + part * 8 + i];
          uint4* d = reinterpret_cast<uint4*>(p.cols + q * p.cols_plane + (c0 + col) * rp + r0 + part * 16);
          d[0] = make_uint4(t[0], t[1], t[2], t[3]);
          d[1] = make_uint4(t[4], t[5], t[6], t[7]);
        }
        __syncthreads();
      }
    }
  }
}

// ---- plans -----------------------------------------------------------------

int64_t ceil64(int64_t v) { return (v + 63) / 64 * 64; }

struct Plan {
  int tile;       // 128 or 64
  int splits;
};

Plan plan_product(int64_t m, int64_t n, int64_t stages) {   // m, n > 0
  const int64_t t128 = ((m + 127) / 128) * ((n + 127) / 128);
  Plan p;
  p.tile = t128 >= 256 ? 128 : 64;
  const int64_t tiles = ((m + p.tile - 1) / p.tile) * ((n + p.tile - 1) / p.tile);
  int64_t s = 512 / tiles;
  if (s > stages / 4) s = stages / 4;
  p.splits = static_cast<int>(s < 1 ? 1 : s);
  return p;
}

int64_t partial_bytes(int64_t m, int64_t n, int64_t stages) {
  if (m == 0 || n == 0) return 0;
  const Plan p = plan_product(m, n, stages);
  return p.splits > 1 ? p.splits * m * n * 4 : 0;
}

// Takes pieces of the workspace, 256-byte aligned; with a null base it only counts.
struct Arena {
  char* base;
  int64_t used = 0;
  template <typename T>
  T* take(int64_t bytes) {
    char* p = base != nullptr ? base + used : nullptr;
    used += (bytes + 255) / 256 * 256;
    return reinterpret_cast<T*>(p);
  }
};

hipError_t run_pack(const Pack& p, hipStream_t stream) {
  const int64_t tiles = ((p.c + 63) / 64) * ((p.r + 63) / 64);
  if (tiles == 0) return hipSuccess;
  pack_kernel<<<static_cast<unsigned>(tiles < (1 << 20) ? tiles : (1 << 20)), 256, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t run_product(Product g, hipStream_t stream) {
  if (g.m == 0 || g.n == 0) return hipSuccess;
  const Plan p = plan_product(g.m, g.n, static_cast<int64_t>(g.nk) * g.terms);
  g.splits = p.splits;
  g.tiles_m = static_cast<int32_t>((g.m + p.tile - 1) / p.tile);
  g.tiles_n = static_cast<int32_t>((g.n + p.tile - 1) / p.tile);
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(g.tiles_m) * g.tiles_n), static_cast<unsigned>(p.splits));
  if (p.tile == 128) tile_kernel<128, 128><<<grid, 256, 0, stream>>>(g);
  else tile_kernel<64, 64><<<grid, 256, 0, stream>>>(g);
  if (p.splits > 1) {
    const int64_t blocks = (g.m * g.n + 255) / 256;
    join_kernel<<<static_cast<unsigned>(blocks < 4096 ? blocks : 4096), 256, 0, stream>>>(g);
  }
  return hipGetLastError();
}

// An operand of a product: where it lies, or the packing that makes it.
struct Operand {
  const __bf16* p;
  int64_t ld, plane;
};

int planes_of(Elem t) { return t == Elem::f32 ? 3 : 1; }
int terms_of(Elem t) { return t == Elem::f32 ? 6 : 1; }
bool direct(Elem t, int64_t k) { return t == Elem::bf16 && k % 64 == 0; }

// The row-major operand (r, c) of a product over c.
Operand rows_operand(const void* src, Elem t, int64_t r, int64_t c, Arena& ws, hipStream_t stream, hipError_t& err) {
  if (direct(t, c)) return {static_cast<const __bf16*>(src), c, 0};
  const int64_t ld = ceil64(c), plane = r * ld;
  __bf16* d = ws.take<__bf16>(planes_of(t) * plane * 2);
  if (ws.base != nullptr && err == hipSuccess) {
    Pack p{};
    p.src = src;
    p.type = t;
    p.r = r;
    p.c = c;
    p.planes = planes_of(t);
    p.rows = d;
    p.rows_plane = plane;
    err = run_pack(p, stream);
  }
  return {d, ld, plane};
}

// The transpose of (r, c) as an operand of a product over r.
Operand cols_operand(const void* src, Elem t, int64_t r, int64_t c, Arena& ws, hipStream_t stream, hipError_t& err) {
  const int64_t ld = ceil64(r), plane = c * ld;
  __bf16* d = ws.take<__bf16>(planes_of(t) * plane * 2);
  if (ws.base != nullptr && err == hipSuccess) {
    Pack p{};
    p.src = src;
    p.type = t;
    p.r = r;
    p.c = c;
    p.planes = planes_of(t);
    p.cols = d;
    p.cols_plane = plane;
    err = run_pack(p, stream);
  }
  return {d, ld, plane};
}

Product product_of(const Operand& a, const Operand& b, Elem t, int64_t m, int64_t n, int64_t k, Arena& ws) {
  Product g{};
  g.a = a.p;
  g.b = b.p;
  g.a_plane = a.plane;
  g.b_plane = b.plane;
  g.lda = a.ld;
  g.ldb = b.ld;
  g.m = m;
  g.n = n;
  g.nk = static_cast<int32_t>((k + 63) / 64);
  g.terms = terms_of(t);
  g.partial = ws.take<float>(partial_bytes(m, n, static_cast<int64_t>(g.nk) * g.terms));
  return g;
}

// The forward's steps; with a null workspace they only count its bytes.
hipError_t linear_steps(const LinearParams& p, Arena& ws, hipStream_t stream) {
  hipError_t err = hipSuccess;
  const Operand a = rows_operand(p.x, p.type, p.rows, p.in, ws, stream, err);
  const Operand b = rows_operand(p.w, p.type, p.out, p.in, ws, stream, err);
  Product g = product_of(a, b, p.type, p.rows, p.out, p.in, ws);
  g.e = {p.bias, p.residual, p.act, p.out_type, p.type, p.y, p.pre};
  if (ws.base == nullptr || err != hipSuccess) return err;
  return run_product(g, stream);
}

hipError_t backward_steps(const LinearBackwardParams& p, bool need_dx, bool need_dw, bool need_db, Arena& ws,
                          hipStream_t stream) {
  hipError_t err = hipSuccess;
  const bool run = ws.base != nullptr;
  const int planes = planes_of(p.type);
  // dz: its rows for dx (dy itself where that serves), its columns for dW, its sums for db
  const bool plain = p.act == Act::none && p.dy_type == p.type && direct(p.type, p.out);
  const int64_t ld_rows = ceil64(p.out), ld_cols = ceil64(p.rows), parts = (p.rows + 63) / 64;
  Pack z{};
  z.src = p.dy;
  z.type = p.dy_type;
  z.pre = p.act == Act::none ? nullptr : p.pre;
  z.pre_type = p.type;
  z.act = p.act;
  z.r = p.rows;
  z.c = p.out;
  z.planes = planes;
  z.rows_plane = p.rows * ld_rows;
  z.cols_plane = p.out * ld_cols;
  if (need_dx && !plain) z.rows = ws.take<__bf16>(planes * z.rows_plane * 2);
  if (need_dw) z.cols = ws.take<__bf16>(planes * z.cols_plane * 2);
  if (need_db) z.sums = ws.take<float>(parts * p.out * 4);
  if (run && (z.rows != nullptr || z.cols != nullptr || z.sums != nullptr)) err = run_pack(z, stream);
  if (run && need_db && err == hipSuccess && p.out > 0)
    err = launch_join_columns(z.sums, parts, p.out, p.out, p.db, nullptr, stream);
  if (need_dx) {
    const Operand a = plain ? Operand{static_cast<const __bf16*>(p.dy), p.out, 0} : Operand{z.rows, ld_rows, z.rows_plane};
    const Operand b = cols_operand(p.w, p.type, p.out, p.in, ws, stream, err);
    Product g = product_of(a, b, p.type, p.rows, p.in, p.out, ws);
    g.e = {nullptr, nullptr, Act::none, p.type, p.type, p.dx, nullptr};
    if (run && err == hipSuccess) err = run_product(g, stream);
  }
  if (need_dw) {
    const Operand a{z.cols, ld_cols, z.cols_plane};
    const Operand b = cols_operand(p.x, p.type, p.rows, p.in, ws, stream, err);
    Product g = product_of(a, b, p.type, p.out, p.in, p.rows, ws);
    g.e = {nullptr, nullptr, Act::none, p.dw_type, p.type, p.dw, nullptr};
    if (run && err == hipSuccess) err = run_product(g, stream);
  }
  return err;
}

}  // namespace

int64_t linear_workspace(Elem type, int64_t rows, int64_t in, int64_t out) {
  LinearParams p{};
  p.type = type;
  p.rows = rows;
  p.in = in;
  p.out = out;
  Arena ws{nullptr};
  (void)linear_steps(p, ws, nullptr);
  return ws.used;
}

hipError_t launch_linear(const LinearParams& p, hipStream_t stream) {
  static char none;
  Arena ws{p.workspace != nullptr ? p.workspace : &none};   // (nothing is taken when no bytes are needed)
  return linear_steps(p, ws, stream);
}

int64_t linear_backward_workspace(Elem type, Elem dy_type, Act act, int64_t rows, int64_t in, int64_t out, bool dx,
                                  bool dw, bool db) {
  LinearBackwardParams p{};
  p.type = type;
  p.dy_type = dy_type;
  p.act = act;
  p.rows = rows;
  p.in = in;
  p.out = out;
  Arena ws{nullptr};
  (void)backward_steps(p, dx, dw, db, ws, nullptr);
  return ws.used;
}

hipError_t launch_linear_backward(const LinearBackwardParams& p, hipStream_t stream) {
  static char none;
  Arena ws{p.workspace != nullptr ? p.workspace : &none};
  return backward_steps(p, p.dx != nullptr, p.dw != nullptr, p.db != nullptr, ws, stream);
}

}  // namespace vn
