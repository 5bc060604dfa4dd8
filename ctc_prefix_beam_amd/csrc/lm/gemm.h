// The matrix product behind the token loss and its gradients:
//   C[m, n] = sum_k A(m, k) B(n, k),   float32 sums,
// with what follows the product done on the sums in registers (the Epilogue).
// Either operand may be stored with k contiguous (row m: k = 0..) or with m
// contiguous (row k: m = 0..), so that the products of the gradients read x, w
// and d as they are, without transposed copies.
//
// A workgroup computes BM x BN from tiles of 128 bytes of k per row (64 16-bit
// values or 32 floats), double-buffered in LDS and filled by loads that go
// straight there, 1 KB per wave instruction.  Such a load writes its 64 pieces
// of 16 bytes one after another, so the layout that spreads LDS reads over all
// banks is made by choosing which piece each lane fetches:
//   k contiguous: piece p of row r is at r*128 + (p ^ ((r >> 1) & 7)) * 16, so
//     that the 16 rows that a 16-byte fragment read touches fill all 256 bytes
//     of the banks once;
//   m contiguous: piece p of k-row k is at k*RB + (p ^ swizzle(k)) * 16, so that
//     the k-rows a fragment read touches lie in different banks.
// Pieces outside the operand are fetched as zeros (an offset past the buffer
// descriptor's range), so sizes need not be multiples of the tile.
#pragma once
#include "common.h"

namespace ctcpb_lm {

constexpr uint32_t kOutside = 0x80000000u;   // beyond every buffer descriptor's range

typedef __attribute__((address_space(3))) char lds_char;

template <typename T>
struct Frag;

template <>
struct Frag<__bf16> {
  typedef bf16x8 V;
  static constexpr int kMfma = 32;   // k of one fragment (over the four lane groups)
  static __device__ f32x4 mac(V a, V b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Frag<_Float16> {
  typedef f16x8 V;
  static constexpr int kMfma = 32;
  static __device__ f32x4 mac(V a, V b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Frag<float> {
  typedef f32x4 V;
  static constexpr int kMfma = 16;
  static __device__ f32x4 mac(V a, V b, f32x4 c) {
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
    return c;
  }
};

// One operand: `rows` along m (or n) and K along k, element (m, k) at
// data[m*ld + k] (k contiguous) or data[k*ld + m] (m contiguous); ld in bytes,
// a multiple of 16, data 16-byte aligned.  Where m is contiguous, every row of
// the operand can be read up to the next multiple of 16 bytes.
struct Operand {
  const char* data;
  int64_t ld;
  int32_t rows;
};

// Fetches an R-row tile of an operand into LDS and reads fragments from it.
// W: waves of the workgroup.
template <typename T, int R, bool KC, int W>
struct TileLoader {
  static constexpr int kBK = 128 / sizeof(T);
  static constexpr int kPer = 16 / sizeof(T);     // elements of a piece
  static constexpr int kLoads = R / 8 / W;        // 1 KB loads per wave
  static constexpr int kRow = KC ? 128 : R * (int)sizeof(T);   // bytes of a row in LDS
  static constexpr int kPieces = kRow / 16;
  static_assert(kLoads * 8 * W == R, "tile and waves do not match");
  typedef typename Frag<T>::V V;

  const char* base;
  int64_t step;            // bytes from one k-tile to the next
  uint32_t off[kLoads];
  int32_t kpos[kLoads];    // first k of the lane's piece in the tile

  static __device__ int swizzle(int k) {
    if constexpr (sizeof(T) == 2)
      return ((k & 3) | ((k >> 3) & 1) << 2) << 1;
    else
      return ((k >> 2) & 3) << 2;
  }

  __device__ void init(const Operand& o, int row0, int wave, int lane) {
    if constexpr (KC) {
      base = o.data + row0 * o.ld;
      step = 128;
    } else {
      base = o.data + (int64_t)row0 * (int)sizeof(T);
      step = kBK * o.ld;
    }
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int i = (wave * kLoads + q) * 64 + lane;   // piece of the tile
      const int r = i / kPieces, p = i % kPieces;
      if constexpr (KC) {
        const int lp = p ^ ((r >> 1) & 7);
        kpos[q] = lp * kPer;
        off[q] = row0 + r < o.rows ? (uint32_t)(r * o.ld + lp * 16) : kOutside;
      } else {
        const int lp = p ^ swizzle(r);
        kpos[q] = r;
        off[q] = row0 + lp * kPer < o.rows ? (uint32_t)(r * o.ld + lp * 16) : kOutside;
      }
    }
  }

  // The tile of k0 .. (of K in all) to `lds`; `base` moves on to the next one.
  __device__ void load(char* lds, int k0, int K, int wave) {
    const bool whole = k0 + kBK <= K;
    __amdgpu_buffer_rsrc_t rsrc =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, 0x7fffffff, 0x00027000);
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      uint32_t o = off[q];
      if (!whole && k0 + kpos[q] >= K) o = kOutside;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rsrc, (lds_char*)(lds + (wave * kLoads + q) * 1024), 16, o, 0, 0, 0);
    }
    base += step;
  }

  // The fragment of rows r0 .. r0+15 (r0 a multiple of 16) and k-step kk.
  static __device__ V read(const char* lds, int r0, int kk, int lane) {
    const int g = lane >> 4, c = lane & 15;
    if constexpr (KC) {
      const int p = (kk * 4 + g) ^ (c >> 1);
      return *reinterpret_cast<const V*>(lds + (r0 + c) * 128 + p * 16);
    } else if constexpr (sizeof(T) == 2) {
      // two transposing reads of four k each: lane i of a group gives the address of
      // four values of k-row i/4 and receives the four k of column i
      typedef short s4 __attribute__((ext_vector_type(4)));
      const int k = kk * 32 + g * 8 + (c >> 2);
      const int p = (r0 / 8 + ((c & 3) >> 1)) ^ swizzle(g * 8 + (c >> 2));
      const char* at = lds + k * kRow + p * 16 + (c & 1) * 8;
      typedef __attribute__((address_space(3))) s4* ptr;
      const s4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(lds_char*)at);
      const s4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(lds_char*)(at + 4 * kRow));
      return __builtin_bit_cast(V, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      V v;
      const int p = (r0 / 4 + (c >> 2)) ^ (g << 2);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = *reinterpret_cast<const float*>(lds + (kk * 16 + g * 4 + j) * kRow + p * 16 +
                                               (c & 3) * 4);
      return v;
    }
  }
};

struct GemmArgs {
  Operand a, b;
  int32_t K;
  int32_t tiles_m, tiles_n;
};

// Tile of workgroup `id`: consecutive ids go to the eight XCDs in turn, so each
// XCD is given a contiguous part of the tiles, walked eight n-tiles wide, to
// find its operands in its own L2.
__device__ inline void tile_of(const GemmArgs& a, int id, int* tm, int* tn) {
  const int total = a.tiles_m * a.tiles_n, per = total / 8;
  if (id < per * 8) id = (id % 8) * per + id / 8;
  const int band = 8 * a.tiles_m;
  const int first = id / band * 8;
  const int wide = min(8, a.tiles_n - first);
  *tn = first + id % band % wide;
  *tm = id % band / wide;
}

// BM x BN per workgroup, WM x WN waves.
template <typename T, int BM, int BN, int WM, int WN, bool AKC, bool BKC, typename Epilogue>
__global__ __launch_bounds__(64 * WM * WN) void gemm_kernel(GemmArgs a, Epilogue ep) {
  constexpr int W = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
  typedef TileLoader<T, BM, AKC, W> LA;
  typedef TileLoader<T, BN, BKC, W> LB;
  __shared__ __align__(1024) char lds[2][(BM + BN) * 128];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  int tm, tn;
  tile_of(a, blockIdx.x, &tm, &tn);
  LA la;
  LB lb;
  la.init(a.a, tm * BM, wave, lane);
  lb.init(a.b, tn * BN, wave, lane);
  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  la.load(lds[0], 0, a.K, wave);
  lb.load(lds[0] + BM * 128, 0, a.K, wave);
  __syncthreads();
  int cur = 0;
  for (int k0 = 0; k0 < a.K; k0 += LA::kBK) {
    if (k0 + LA::kBK < a.K) {
      la.load(lds[cur ^ 1], k0 + LA::kBK, a.K, wave);
      lb.load(lds[cur ^ 1] + BM * 128, k0 + LA::kBK, a.K, wave);
    }
    const char *ta = lds[cur], *tb = lds[cur] + BM * 128;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      typename Frag<T>::V fa[TM], fb[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i) fa[i] = LA::read(ta, (wm * TM + i) * 16, kk, lane);
#pragma unroll
      for (int j = 0; j < TN; ++j) fb[j] = LB::read(tb, (wn * TN + j) * 16, kk, lane);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = Frag<T>::mac(fa[i], fb[j], acc[i][j]);
    }
    __syncthreads();
    cur ^= 1;
  }
  // sums acc[i][j][r]: m = tm*BM + (wm*TM + i)*16 + (lane>>4)*4 + r, n = tn*BN + (wn*TN + j)*16 + (lane&15)
  ep.template run<TM, TN, WM, WN>(acc, tm, tn, wm, wn, lane, lds[0]);
}

}  // namespace ctcpb_lm
