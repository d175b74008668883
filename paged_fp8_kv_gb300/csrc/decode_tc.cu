// The swap-AB decode kernel on plain scores (see decode_tc.cuh), the TMA
// descriptors of the pools, and the verification hooks' kernels.

#include <cuda.h>
#include <cuda_runtime.h>

#include "decode_tc.cuh"

namespace mj {
// -------------------------------------------------------- host: tensor maps

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  }
  return fn;
}

}  // namespace

// (d bytes, rows in page, kv heads, pages) view of a paged e4m3 pool; one box
// is box_rows rows of box_heads heads: 128 bytes x box_rows x box_heads,
// head-major in shared memory, 128-byte swizzle.
bool make_kv_map(CUtensorMap* m, const uint8_t* base, int page_size, int h_k, int num_pages, int64_t s_row,
                 int64_t s_head, int64_t s_page, int box_rows, int box_heads, int kv_format) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[4] = {128, static_cast<cuuint64_t>(page_size), static_cast<cuuint64_t>(h_k),
                              static_cast<cuuint64_t>(num_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(s_row), static_cast<cuuint64_t>(s_head),
                                 static_cast<cuuint64_t>(s_page)};
  const cuuint32_t box[4] = {128, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(box_heads), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUtensorMapDataType type = kv_format == 0   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : kv_format == 3 ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B
                                                    : CU_TENSOR_MAP_DATA_TYPE_16U6_ALIGN16B;
  const CUresult r = enc(m, type, 4, const_cast<uint8_t*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// nvfp4 pools as byte tensors: the codes (64 bytes a row) and the scale
// plane (a page's rows of one head, PS x 8 bytes, seen as PS / 16 rows of
// 128 bytes); one box is one page of one head, unswizzled.
bool make_nv_map(CUtensorMap* m, const uint8_t* base, bool scales, int page_size, int h_k, int num_pages,
                 int64_t s_row, int64_t s_head, int64_t s_page) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t inner = scales ? 128 : 64;
  const cuuint64_t rows = scales ? static_cast<cuuint64_t>(page_size / 16) : static_cast<cuuint64_t>(page_size);
  const cuuint64_t dims[4] = {inner, rows, static_cast<cuuint64_t>(h_k), static_cast<cuuint64_t>(num_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(scales ? 128 : s_row), static_cast<cuuint64_t>(s_head),
                                 static_cast<cuuint64_t>(s_page)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(inner), static_cast<cuuint32_t>(rows), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

namespace {

template <int R>
cudaError_t launch_tc_q(const DecodeDev& a, int n_q_tiles, bool q_e4m3, cudaStream_t stream) {
  if (a.kv_format == 4) {  // nvfp4: e4m3 Q, up to 32 rows (validated before)
    if constexpr (R <= 32) {
      if (q_e4m3) return launch_tc<R, true, true, false>(a, n_q_tiles, stream);
    }
    return cudaErrorInvalidValue;
  }
  return q_e4m3 ? launch_tc<R, true, false, false>(a, n_q_tiles, stream) : launch_tc<R, false, false, false>(a, n_q_tiles, stream);
}

// ---------------------------------------------------------------- checks
// The producer's page gather and the CUDA-core kernel's dequant as
// standalone launches, so that tests can compare them byte- and bit-exact
// with the oracle: the same tensor maps (make_kv_map), the same page lookup
// (lane j fetches page j of a 128-row tile through the block table; pages
// past the sequence end are fetched out of range, as zeros), the same TMA
// boxes, and the 128-byte swizzle the MMA descriptors assume, undone here.

// grid (tiles, h_k, num_seqs), 64 threads; out rows [b][g][row][128 bytes]
__global__ void __launch_bounds__(64) gather_kv_kernel(const DecodeDev a, const __grid_constant__ CUtensorMap tmap,
                                                       uint8_t* __restrict__ out, int out_rows) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tile = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t tile_s = ptx::smem_u32(tile);
  const uint32_t bar = tile_s + kKVTileBytes;
  const int t = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int L = a.seq_lens[b];
  const int T = L > 0 ? (L + kTileKV - 1) / kTileKV : 1;
  if (t >= T) return;  // uniform over the CTA
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) {
    ptx::mbar_init(bar, 1);
    ptx::fence_mbar_init();
  }
  __syncthreads();
  if (tid < 32) {
    const int PS = a.page_size;
    const int ppt = kTileKV / PS;
    int valid_pages = (L + PS - 1) / PS;
    valid_pages = valid_pages < a.max_blocks ? valid_pages : a.max_blocks;
    const int blk = t * ppt + lane;
    const int page = (lane < ppt && blk < valid_pages)
                         ? a.block_table[static_cast<int64_t>(b) * a.max_blocks + blk]
                         : a.num_pages;
    if (lane == 0) ptx::mbar_arrive_expect_tx(bar, kv_box_bytes(a.kv_format, kTileKV));
    __syncwarp();
    if (lane < ppt) ptx::tma_load_4d(tile_s + lane * PS * 128, &tmap, bar, 0, 0, g, page);
  }
  volatile int never = 0;
  if (!ptx::mbar_wait_bounded(bar, 0, &never, kWaitNs)) {  // rows stay unwritten: the test fails
    ptx::mbar_wait_bounded(bar, 0, &never, kWaitNs / 4);     // (a bounded drain before leaving)
    return;
  }
  for (int i = tid; i < kTileKV * 8; i += 64) {
    const int r = i >> 3, cc = i & 7;
    const int key = t * kTileKV + r;
    if (key >= L || key >= out_rows) continue;
    const uint4 v = *reinterpret_cast<const uint4*>(tile + r * 128 + ((cc ^ (r & 7)) << 4));
    *reinterpret_cast<uint4*>(out + ((static_cast<int64_t>(b) * a.h_k + g) * out_rows + key) * 128 + cc * 16) = v;
  }
}

// 64 threads: codes 4t .. 4t + 3 through the CUDA-core kernel's conversion
__global__ void dequant_e4m3_kernel(float* __restrict__ out) {
  const uint32_t c0 = 4u * threadIdx.x;
  const uint32_t w = c0 | ((c0 + 1) << 8) | ((c0 + 2) << 16) | ((c0 + 3) << 24);
  float v[4];
  e4m3x4_to_f32(w, v);
#pragma unroll
  for (int k = 0; k < 4; ++k) out[c0 + k] = v[k];
}

// The bounded-wait primitive on its own: one warp waits on an mbarrier that
// nothing arrives on, so the wait must give up after `limit_ns`; the warp then
// reports MJ_ERR_TIMEOUT in the status word, as the decode kernels do, and the
// time it waited.  No other warp and no named barrier is involved, so the
// launch ends whatever the primitive does with its limit.
__global__ void bounded_wait_kernel(int32_t* status, int64_t* waited_ns, uint64_t limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int abort_flag;
  const uint32_t b = ptx::smem_u32(&bar);
  if (threadIdx.x == 0) {
    ptx::mbar_init(b, 1);
    abort_flag = 0;
    ptx::fence_mbar_init();
  }
  __syncwarp();
  const uint64_t t0 = ptx::globaltimer_ns();
  const bool done = ptx::mbar_wait_bounded(b, 0, &abort_flag, limit_ns);
  const uint64_t t1 = ptx::globaltimer_ns();
  if (threadIdx.x == 0) {
    if (!done) atomicExch(status, 5);  // MJ_ERR_TIMEOUT
    if (waited_ns) *waited_ns = static_cast<int64_t>(t1 - t0);
  }
}

}  // namespace

cudaError_t launch_bounded_wait(int32_t* status, int64_t* waited_ns, uint64_t limit_ns, cudaStream_t stream) {
  bounded_wait_kernel<<<1, 32, 0, stream>>>(status, waited_ns, limit_ns);
  return cudaGetLastError();
}

// nvfp4 pools: rows 0 .. L - 1 converted to e4m3 by the decode kernel's
// conversion (nvfp4_group_to_e4m3), codes and scales read through the block
// table with plain loads; grid (tiles, h_k, num_seqs), 128 threads.
__global__ void __launch_bounds__(128) gather_nvfp4_kernel(const DecodeDev a, bool values, uint8_t* __restrict__ out,
                                                           int out_rows) {
  const int t = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int L = a.seq_lens[b];
  const uint8_t* pool = values ? a.v : a.k;
  const uint8_t* scales = values ? a.vs : a.ks;
  const int64_t p_page = values ? a.v_page : a.k_page, p_row = values ? a.v_row : a.k_row;
  const int64_t p_head = values ? a.v_head : a.k_head;
  const int64_t s_page = values ? a.vs_page : a.ks_page, s_head = values ? a.vs_head : a.ks_head;
  for (int j = threadIdx.x; j < kTileKV * 8; j += 128) {
    const int key = t * kTileKV + (j >> 3), cc = j & 7;
    if (key >= L || key >= out_rows) continue;
    const int page = a.block_table[static_cast<int64_t>(b) * a.max_blocks + key / a.page_size];
    const int row = key % a.page_size;
    const uint2 c = *reinterpret_cast<const uint2*>(pool + page * p_page + row * p_row + g * p_head + cc * 8);
    const uint32_t sc = scales[page * s_page + g * s_head + row * 8 + cc];
    *reinterpret_cast<uint4*>(out + ((static_cast<int64_t>(b) * a.h_k + g) * out_rows + key) * 128 + cc * 16) =
        nvfp4_group_to_e4m3(c, sc);
  }
}

cudaError_t launch_gather_kv(const DecodeDev& a, bool values, uint8_t* out, int out_rows, cudaStream_t stream) {
  if (a.kv_format == 4) {
    const int tiles = (out_rows + kTileKV - 1) / kTileKV;
    dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(a.h_k), static_cast<unsigned>(a.num_seqs));
    gather_nvfp4_kernel<<<grid, 128, 0, stream>>>(a, values, out, out_rows);
    return cudaGetLastError();
  }
  CUtensorMap m;
  const bool ok = values ? make_kv_map(&m, a.v, a.page_size, a.h_k, a.num_pages, a.v_row, a.v_head, a.v_page,
                                       a.page_size, 1, a.kv_format)
                         : make_kv_map(&m, a.k, a.page_size, a.h_k, a.num_pages, a.k_row, a.k_head, a.k_page,
                                       a.page_size, 1, a.kv_format);
  if (!ok) return cudaErrorInvalidValue;
  const int tiles = (out_rows + kTileKV - 1) / kTileKV;
  const int smem = kKVTileBytes + 1024 + 64;  // tile, alignment slack, mbarrier
  dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(a.h_k), static_cast<unsigned>(a.num_seqs));
  gather_kv_kernel<<<grid, 64, smem, stream>>>(a, m, out, out_rows);
  return cudaGetLastError();
}

cudaError_t launch_dequant_e4m3(float* out, cudaStream_t stream) {
  dequant_e4m3_kernel<<<1, 64, 0, stream>>>(out);
  return cudaGetLastError();
}

cudaError_t launch_decode_tc(const DecodeDev& a, int rows_per_cta, int n_q_tiles, bool q_e4m3,
                             cudaStream_t stream) {
  switch (rows_per_cta) {
    case 8: return launch_tc_q<8>(a, n_q_tiles, q_e4m3, stream);
    case 16: return launch_tc_q<16>(a, n_q_tiles, q_e4m3, stream);
    case 32: return launch_tc_q<32>(a, n_q_tiles, q_e4m3, stream);
    case 64: return launch_tc_q<64>(a, n_q_tiles, q_e4m3, stream);
    default: return cudaErrorInvalidValue;
  }
}

int tc_min_blocks(int rows_per_cta, bool q_e4m3, bool nvfp4) {
  if (nvfp4) return 1;
  switch (rows_per_cta) {
    case 8: return q_e4m3 ? TcCfg<8, true>::kMinBlocks : TcCfg<8, false>::kMinBlocks;
    case 16: return q_e4m3 ? TcCfg<16, true>::kMinBlocks : TcCfg<16, false>::kMinBlocks;
    case 32: return q_e4m3 ? TcCfg<32, true>::kMinBlocks : TcCfg<32, false>::kMinBlocks;
    case 64: return q_e4m3 ? TcCfg<64, true>::kMinBlocks : TcCfg<64, false>::kMinBlocks;
    default: return 1;
  }
}

int tc_smem_bytes(int rows_per_cta, bool q_e4m3, bool nvfp4) {
  if (nvfp4) {
    switch (rows_per_cta) {
      case 8: return TcCfg<8, true, true>::kBytes;
      case 16: return TcCfg<16, true, true>::kBytes;
      case 32: return TcCfg<32, true, true>::kBytes;
      default: return 0;
    }
  }
  switch (rows_per_cta) {
    case 8: return q_e4m3 ? TcCfg<8, true>::kBytes : TcCfg<8, false>::kBytes;
    case 16: return q_e4m3 ? TcCfg<16, true>::kBytes : TcCfg<16, false>::kBytes;
    case 32: return q_e4m3 ? TcCfg<32, true>::kBytes : TcCfg<32, false>::kBytes;
    case 64: return q_e4m3 ? TcCfg<64, true>::kBytes : TcCfg<64, false>::kBytes;
    default: return 0;
  }
}

}  // namespace mj
