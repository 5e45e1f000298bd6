// blocknorm_api.cu -- the C ABI of the norms around a block (declared in
// include/libnorm.h): argument checks, workspace layout, then dispatch.  The
// kernels live in blocknorm_<dtype>.cu.
#include "blocknorm.h"
#include "heads_check.h"

namespace nrm {
namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxCols = int64_t(1) << 27;  // grids of 32 columns, and partial rows of up to 2^40 bytes

nrm_status check_block(int64_t rows, int64_t cols, int64_t gates, nrm_dtype dt) {
    if (dt != NRM_F32 && dt != NRM_F16 && dt != NRM_BF16)
        return fail(NRM_ERR_INVALID_ARG, "unknown dtype %d", int(dt));
    if (rows < 0) return fail(NRM_ERR_INVALID_ARG, "rows must be >= 0");
    if (cols < 1) return fail(NRM_ERR_INVALID_ARG, "cols must be >= 1");
    if (cols > kMaxCols) return fail(NRM_ERR_UNSUPPORTED, "cols must be <= 2^27");
    if (rows > kMaxElems / cols) return fail(NRM_ERR_UNSUPPORTED, "rows*cols must be <= 2^40");
    if (gates < 0 || (gates > 0 && (rows % gates || (rows == 0 && gates > kMaxElems / cols))))
        return fail(NRM_ERR_INVALID_ARG, "gates must divide rows");
    return NRM_OK;
}

// The chunks of rows whose column sums are kept apart, and the workspace's bytes.
int64_t block_chunks(const DevInfo& dev, int64_t rows) { return std::min<int64_t>(rows, block_max_chunks(dev)); }
size_t block_bytes(const DevInfo& dev, int64_t rows, int64_t cols) {
    return size_t((rows + 3) / 4 * 4 + 4 * block_chunks(dev, rows) * cols) * 4;
}

nrm_status check_params(std::initializer_list<const void*> ptrs, nrm_dtype dt) {
    for (const void* p : ptrs)
        if (!aligned(p, dsize(dt))) return fail(NRM_ERR_INVALID_ARG, "pointers must be aligned to their element size");
    return NRM_OK;
}

// Rows of whole 16-byte vectors at aligned addresses.
bool whole_vectors(std::initializer_list<const void*> ptrs, int64_t cols, nrm_dtype dt) {
    if (cols * int64_t(dsize(dt)) % 16) return false;
    for (const void* p : ptrs)
        if (!aligned(p, 16)) return false;
    return true;
}

}  // namespace
}  // namespace nrm

using namespace nrm;

extern "C" {

nrm_status nrm_block_norm_fwd(const void* x, const void* f, const void* gate, const void* w_post, const void* w_pre,
                              void* y, void* h, float* rstd_post, float* rstd_pre, int64_t rows, int64_t cols,
                              int64_t gates, float alpha, float eps, int post, nrm_dtype dt, nrm_stream_t stream) {
    return entry([&]() -> nrm_status {
        NRM_TRY(check_block(rows, cols, gates, dt));
        NRM_TRY(check_eps(eps));
        if (!std::isfinite(alpha)) return fail(NRM_ERR_INVALID_ARG, "alpha must be finite");
        if (!post) w_post = nullptr, rstd_post = nullptr;
        if (!h) w_pre = nullptr, rstd_pre = nullptr;
        if (rows > 0 && (!x || !f || !y)) return fail(NRM_ERR_INVALID_ARG, "x, f and y must not be NULL");
        if (rows > 0 && (gate != nullptr) != (gates > 0))
            return fail(NRM_ERR_INVALID_ARG, "gate is NULL exactly when gates is 0");
        NRM_TRY(check_params({x, f, gate, w_post, w_pre, y, h}, dt));
        NRM_TRY(check_stats({rstd_post, rstd_pre}, 4));
        if (rows > 0 && (y == f || (h && (h == x || h == y))))
            return fail(NRM_ERR_INVALID_ARG, "y may be x and h may be f, no other overlap");
        if (rstd_post && rstd_post == rstd_pre)
            return fail(NRM_ERR_INVALID_ARG, "rstd_post and rstd_pre are the same memory");
        BlockArgs a{};
        a.x = x;
        a.f = f;
        a.gate = gate;
        a.w_post = w_post;
        a.w_pre = w_pre;
        a.y = y;
        a.h = h;
        a.rstd_post = rstd_post;
        a.rstd_pre = rstd_pre;
        a.rows = rows;
        a.cols = int(cols);
        a.gates = rows > 0 ? gates : 0;
        a.per_gate = make_row_div(a.gates ? rows / gates : 1, rows);
        a.alpha = alpha;
        a.eps = eps;
        a.post = post != 0;
        const bool vec = whole_vectors({x, f, gate, w_post, w_pre, y, h}, cols, dt);
        return by_dtype(dt, [&](auto tag) {
            return block_norm_fwd<decltype(tag)>(a, vec, reinterpret_cast<cudaStream_t>(stream));
        });
    });
}

size_t nrm_block_norm_workspace_bytes(int64_t rows, int64_t cols, int64_t gates, nrm_dtype dt) {
    clear_error();
    const DevInfo* dev = dev_info();
    if (!dev || check_block(rows, cols, gates, dt) != NRM_OK) return 0;
    return std::max<size_t>(block_bytes(*dev, rows, cols), 16);
}

nrm_status nrm_block_norm_bwd(const void* dh, const void* dy, const void* f, const void* y, const void* gate,
                              const void* w_post, const void* w_pre, const float* rstd_post, const float* rstd_pre,
                              void* dx, void* df, void* dgate, void* dw_post, void* dw_pre, int64_t rows,
                              int64_t cols, int64_t gates, float alpha, int post, nrm_dtype dt, void* workspace,
                              size_t workspace_bytes, nrm_stream_t stream) {
    return entry([&]() -> nrm_status {
        NRM_TRY(check_block(rows, cols, gates, dt));
        if (!std::isfinite(alpha)) return fail(NRM_ERR_INVALID_ARG, "alpha must be finite");
        if (!post && dw_post) return fail(NRM_ERR_INVALID_ARG, "dw_post without the norm after the block");
        if (!gates && dgate) return fail(NRM_ERR_INVALID_ARG, "dgate without a gate");
        if (rows > 0 && !dh && dw_pre) return fail(NRM_ERR_INVALID_ARG, "dw_pre without dh");
        if (!post) w_post = nullptr, rstd_post = nullptr;
        if (rows > 0 && !dh) w_pre = nullptr, rstd_pre = nullptr;
        if (rows > 0) {
            if (!dh && !dy) return fail(NRM_ERR_INVALID_ARG, "dh and dy must not both be NULL");
            if (!f || (dh && !y) || !dx || !df) return fail(NRM_ERR_INVALID_ARG, "f, y, dx and df must not be NULL");
            if ((post && !rstd_post) || (dh && !rstd_pre))
                return fail(NRM_ERR_INVALID_ARG, "the saved statistics must not be NULL");
            if ((gate != nullptr) != (gates > 0))
                return fail(NRM_ERR_INVALID_ARG, "gate is NULL exactly when gates is 0");
            for (const void* in : {dh, dy, f, y})
                if (dx == in || df == in) return fail(NRM_ERR_INVALID_ARG, "dx and df must not be an input");
            if (dx == df) return fail(NRM_ERR_INVALID_ARG, "dx and df are the same memory");
        }
        if ((dw_post && (dw_post == dw_pre || dw_post == dgate)) || (dw_pre && dw_pre == dgate))
            return fail(NRM_ERR_INVALID_ARG, "two gradients of weights are the same memory");
        NRM_TRY(check_params({dh, dy, f, y, gate, w_post, w_pre, dx, df, dgate, dw_post, dw_pre}, dt));
        NRM_TRY(check_stats({rstd_post, rstd_pre}, 4));
        const DevInfo* dev = dev_info();
        if (!dev) return fail(NRM_ERR_CUDA, "no usable CUDA device");
        BlockArgs a{};
        if (rows > 0 && (dgate || dw_post || dw_pre)) {
            const size_t need = block_bytes(*dev, rows, cols);
            if (!workspace || !aligned(workspace, 16))
                return fail(NRM_ERR_WORKSPACE, "workspace must be non-NULL and 16-byte aligned");
            if (workspace_bytes < need)
                return fail(NRM_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed",
                            workspace_bytes, need);
            a.c2 = static_cast<float*>(workspace);
            a.part = a.c2 + (rows + 3) / 4 * 4;
        }
        a.dh = dh;
        a.dy = dy;
        a.f = f;
        a.y = const_cast<void*>(y);
        a.gate = gate;
        a.w_post = w_post;
        a.w_pre = w_pre;
        a.rstd_post = const_cast<float*>(rstd_post);
        a.rstd_pre = const_cast<float*>(rstd_pre);
        a.dx = dx;
        a.df = df;
        a.dgate = dgate;
        a.dw_post = dw_post;
        a.dw_pre = dw_pre;
        a.rows = rows;
        a.cols = int(cols);
        a.gates = gates;
        a.per_gate = make_row_div(gates > 0 && rows > 0 ? rows / gates : 1, rows);
        a.alpha = alpha;
        a.post = post != 0;
        a.chunks = block_chunks(*dev, rows);
        const bool vec = whole_vectors({dh, dy, f, y, gate, w_post, w_pre, dx, df, dgate}, cols, dt);
        const bool copies = aligned(dh, 16) && aligned(dy, 16) && aligned(f, 16) && aligned(y, 16);
        return by_dtype(dt, [&](auto tag) {
            return block_norm_bwd<decltype(tag)>(a, vec, copies, reinterpret_cast<cudaStream_t>(stream));
        });
    });
}

}  // extern "C"
