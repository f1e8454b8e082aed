// gemm.cu -- the matrix product behind the decoder layers: a plain tiled product
// in fp32 for every layout, type and alignment.
#include "gemm.cuh"

namespace gs {
namespace {

constexpr int kTileMN = 64;
constexpr int kTileK = 16;

struct SimpleParams {
    GemmCall c;
};

// 16 x 16 threads, each 4 x 4 of a 64 x 64 tile.
__device__ void tile_product(const GemmCall& c, const GemmFactor& a, const GemmFactor& b, int64_t m0, int64_t n0,
                             float (&acc)[4][4], float (*sa)[kTileMN + 1], float (*sb)[kTileMN + 1])
{
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    for (int64_t k0 = 0; k0 < c.k; k0 += kTileK) {
        __syncthreads();
        for (int i = threadIdx.x; i < kTileMN * kTileK; i += 256) {
            const int r = a.k_fast ? i / kTileK : i % kTileMN, k = a.k_fast ? i % kTileK : i / kTileMN;
            const int64_t row = m0 + r, kk = k0 + k;
            sa[k][r] = row < c.m && kk < c.k ? load_elem(a.p, a.k_fast ? row * a.ld + kk : kk * a.ld + row, c.type) : 0.0f;
        }
        for (int i = threadIdx.x; i < kTileMN * kTileK; i += 256) {
            const int r = b.k_fast ? i / kTileK : i % kTileMN, k = b.k_fast ? i % kTileK : i / kTileMN;
            const int64_t row = n0 + r, kk = k0 + k;
            sb[k][r] = row < c.n && kk < c.k ? load_elem(b.p, b.k_fast ? row * b.ld + kk : kk * b.ld + row, c.type) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < kTileK; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = __fmaf_rn(sa[k][ty + 16 * i], sb[k][tx + 16 * j], acc[i][j]);
    }
}

__global__ void __launch_bounds__(256) gemm_simple_kernel(const SimpleParams p)
{
    __shared__ float sa[kTileK][kTileMN + 1], sb[kTileK][kTileMN + 1];
    const GemmCall& c = p.c;
    const int64_t tiles_n = (c.n + kTileMN - 1) / kTileMN;
    const int64_t m0 = (int64_t)blockIdx.x / tiles_n * kTileMN, n0 = (int64_t)blockIdx.x % tiles_n * kTileMN;
    const int which = blockIdx.y;
    float acc[4][4] = {}, acc2[4][4] = {};
    if (c.kind == GemmKind::kTwo) tile_product(c, c.a[which], c.b[which], m0, n0, acc, sa, sb);
    else {
        tile_product(c, c.a[0], c.b[0], m0, n0, acc, sa, sb);
        if (c.kind == GemmKind::kSum) tile_product(c, c.a[1], c.b[1], m0, n0, acc, sa, sb);
        if (c.kind == GemmKind::kGlu) tile_product(c, c.a[0], c.b[1], m0, n0, acc2, sa, sb);
    }
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m >= c.m || n >= c.n) continue;
            float v = acc[i][j];
            const float xs = c.x_scale ? c.x_scale[m] : 1.0f;
            if (c.w_scale[0]) v *= xs * c.w_scale[0][n];
            else v *= xs;
            if (c.kind == GemmKind::kGlu) {
                float u = acc2[i][j] * (c.w_scale[1] ? xs * c.w_scale[1][n] : xs);
                if (c.z) {
                    store_elem(c.z, m * c.ldz + n, c.z_type, v);
                    store_elem(c.z2, m * c.ldz2 + n, c.z_type, u);
                }
                v = act_value(v, c.act) * u;
            } else {
                if (c.bias) v += load_elem(c.bias, n, c.bias_type);
                if (c.z) store_elem(c.z, m * c.ldz + n, c.z_type, v);
                v = act_value(v, c.act);
                if (c.residual) v += load_elem(c.residual, m * c.ldr + n, c.out_type);
            }
            store_elem(which ? c.y2 : c.y, m * (which ? c.ldy2 : c.ldy) + n, c.out_type, v);
        }
}

}  // namespace

gs_status gemm_ws_bytes(const GemmCall& c, size_t* bytes)
{
    *bytes = 0;
    return GS_OK;
}

gs_status gemm_run(const GemmCall& c, void* ws, cudaStream_t st)
{
    const int64_t tiles = ((c.m + kTileMN - 1) / kTileMN) * ((c.n + kTileMN - 1) / kTileMN);
    if (tiles > 0x7fffffffll) return GS_ERR_INVALID_ARG;
    SimpleParams p{c};
    gemm_simple_kernel<<<dim3((unsigned)tiles, c.kind == GemmKind::kTwo ? 2 : 1), 256, 0, st>>>(p);
    GS_LAUNCH_CHECK();
    return GS_OK;
}

}  // namespace gs
