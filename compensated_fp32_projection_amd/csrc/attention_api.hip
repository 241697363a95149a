// C ABI of the attention and cache calls (declared in include/cfp32.h):
// argument validation, the device check and workspace sizes.  Every call
// validates all of its arguments before it enqueues anything.
#include "api_checks.h"

namespace {

using namespace cfp32;

// A pool that is written (pages must not overlap) or only read.
bool pool_ok(const void *k, int64_t kp, int64_t kh, int64_t kt, const void *v, int64_t vp, int64_t vh, int64_t vt,
             int64_t P, int64_t Hkv, int64_t page, int64_t D, int kv_type, bool written)
{
    if (!k || !v) return false;
    const size_t a = kv_type == CFP32_KV_F16 ? 2 : 4;
    if (!aligned_to(k, a) || !aligned_to(v, a)) return false;
    if (!view_ok(P, kp, Hkv, kh, page, kt, D) || !view_ok(P, vp, Hkv, vh, page, vt, D)) return false;
    return !written || (distinct_ok(P, kp, Hkv, kh, page, kt, D) && distinct_ok(P, vp, Hkv, vh, page, vt, D));
}

cfp32::Pool make_pool(void *k, int64_t kp, int64_t kh, int64_t kt, void *v, int64_t vp, int64_t vh, int64_t vt,
                      int64_t P, int64_t page, int64_t Hkv, int64_t D, int kv_type)
{
    return {{k, kp, kh, kt}, {v, vp, vh, vt}, (int)P, page_log2(page), (int)Hkv, (int)D, kv_type == CFP32_KV_F16 ? 2 : 4};
}

}  // namespace

extern "C" {

size_t cfp32_attention_prompt_workspace_bytes(int64_t S, int64_t Tk, int64_t Hkv, int64_t D, int kv_type)
{
    if (!size_ok(S) || Tk < 0 || Tk > kMaxKeys || !heads_ok(Hkv, Hkv, D) || !type_ok(kv_type)) return 0;
    if (S == 0 || Tk == 0 || Hkv == 0 || D == 0) return 0;
    if (Hkv > (kMaxDim >> 12) / (Tk / 64 + S)) return 0;
    const size_t n = cfp32::attention_prompt_workspace(S, Tk, Hkv, D, kv_type == CFP32_KV_F16);
    return n ? n + kAlign : 0;
}

cfp32_status cfp32_attention_prompt(const float *q, int64_t q_tok, int64_t q_head, const void *k, int64_t k_tok,
                                    int64_t k_head, const void *v, int64_t v_tok, int64_t v_head, int kv_type,
                                    const int32_t *cu_q, const int32_t *cu_k, float *out, int64_t out_tok,
                                    int64_t out_head, int64_t S, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv,
                                    int64_t D, int causal, double scale, void *workspace, size_t workspace_bytes,
                                    void *stream)
{
    if (!size_ok(S) || !size_ok(Tq) || Tk < 0 || Tk > kMaxKeys || !heads_ok(Hq, Hkv, D) || !type_ok(kv_type))
        return CFP32_ERR_INVALID_VALUE;
    if (S == 0 || Tq == 0 || Hq == 0 || D == 0) return CFP32_OK;
    if (!q || !out || !cu_q || !cu_k || (Tk > 0 && (!k || !v))) return CFP32_ERR_INVALID_VALUE;
    const size_t ka = kv_type == CFP32_KV_F16 ? 2 : 4;
    if (!aligned_to(q, 4) || !aligned_to(out, 4) || !aligned_to(k, ka) || !aligned_to(v, ka))
        return CFP32_ERR_INVALID_VALUE;
    if (!view_ok(Tq, q_tok, Hq, q_head, 1, 0, D) || !view_ok(Tk, k_tok, Hkv, k_head, 1, 0, D) ||
        !view_ok(Tk, v_tok, Hkv, v_head, 1, 0, D) || !view_ok(Tq, out_tok, Hq, out_head, 1, 0, D) ||
        !distinct_ok(Tq, out_tok, Hq, out_head, 1, 0, D))
        return CFP32_ERR_INVALID_VALUE;
    if (!scale_ok(scale)) return CFP32_ERR_INVALID_VALUE;
    if (Tk > 0 && Hkv > (kMaxDim >> 12) / (Tk / 64 + S)) return CFP32_ERR_INVALID_VALUE;
    const size_t need = cfp32_attention_prompt_workspace_bytes(S, Tk, Hkv, D, kv_type);
    if (need && (!workspace || workspace_bytes < need)) return CFP32_ERR_INVALID_VALUE;
    cfp32_status st = api_check_device();
    if (st != CFP32_OK) return st;
    const cfp32::PromptArgs a = {{q, q_tok, q_head}, {k, k_tok, k_head}, {v, v_tok, v_head}, out, out_tok, out_head,
                                 cu_q, cu_k, (int)S, (int)Tq, (int)Tk, (int)Hq, (int)Hkv, (int)D,
                                 kv_type == CFP32_KV_F16, causal != 0, (float)scale};
    return api_launched(cfp32::launch_attention_prompt(a, align_up(workspace), (hipStream_t)stream));
}

size_t cfp32_attention_decode_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t W, int64_t page,
                                              int64_t shared_pages, int kv_type)
{
    const int lg = page_log2(page);
    if (!size_ok(B) || !heads_ok(Hq, Hkv, D) || !size_ok(W) || lg < 0 || W > (kMaxKeys >> lg) || !type_ok(kv_type) ||
        shared_pages < 0 || shared_pages > W)
        return 0;
    if (B == 0 || Hq == 0 || D == 0 || B > (kMaxDim >> 20) / Hq) return 0;
    const size_t n = cfp32::attention_decode_workspace(B, Hq, Hkv, D, W, lg, shared_pages, kv_type == CFP32_KV_F16);
    return n ? n + kAlign : 0;
}

cfp32_status cfp32_attention_decode(const float *q, int64_t q_seq, int64_t q_head, const void *k_pages, int64_t k_page,
                                    int64_t k_head, int64_t k_tok, const void *v_pages, int64_t v_page,
                                    int64_t v_head, int64_t v_tok, int kv_type, int64_t P, int64_t page,
                                    const int32_t *table, int64_t ld_table, int64_t W, const int32_t *lens,
                                    int64_t shared_pages, float *out, int64_t out_seq, int64_t out_head, int64_t B,
                                    int64_t Hq, int64_t Hkv, int64_t D, double scale, void *workspace,
                                    size_t workspace_bytes, void *stream)
{
    const int lg = page_log2(page);
    if (!size_ok(B) || !heads_ok(Hq, Hkv, D) || !size_ok(W) || !size_ok(P) || lg < 0 || W > (kMaxKeys >> lg) ||
        !type_ok(kv_type) || shared_pages < 0 || shared_pages > W)
        return CFP32_ERR_INVALID_VALUE;
    if (B == 0 || Hq == 0 || D == 0) return CFP32_OK;
    if (B > (kMaxDim >> 20) / Hq) return CFP32_ERR_INVALID_VALUE;
    if (!q || !out || !lens || !table_ok(table, ld_table, B, W, true)) return CFP32_ERR_INVALID_VALUE;
    if (P > 0 && !pool_ok(k_pages, k_page, k_head, k_tok, v_pages, v_page, v_head, v_tok, P, Hkv, page, D, kv_type, false))
        return CFP32_ERR_INVALID_VALUE;
    if (!aligned_to(q, 4) || !aligned_to(out, 4) || !view_ok(B, q_seq, Hq, q_head, 1, 0, D) ||
        !view_ok(B, out_seq, Hq, out_head, 1, 0, D) || !distinct_ok(B, out_seq, Hq, out_head, 1, 0, D))
        return CFP32_ERR_INVALID_VALUE;
    if (!scale_ok(scale)) return CFP32_ERR_INVALID_VALUE;
    const size_t need = cfp32_attention_decode_workspace_bytes(B, Hq, Hkv, D, W, page, shared_pages, kv_type);
    if (need && (!workspace || workspace_bytes < need)) return CFP32_ERR_INVALID_VALUE;
    cfp32_status st = api_check_device();
    if (st != CFP32_OK) return st;
    const cfp32::DecodeArgs a = {q, q_seq, q_head,
                                 {const_cast<void *>(k_pages), k_page, k_head, k_tok},
                                 {const_cast<void *>(v_pages), v_page, v_head, v_tok},
                                 table, ld_table, lens, out, out_seq, out_head, (int)B, (int)Hq, (int)Hkv, (int)D,
                                 (int)P, lg, (int)W, (int)shared_pages, kv_type == CFP32_KV_F16, (float)scale};
    return api_launched(cfp32::launch_attention_decode(a, align_up(workspace), (hipStream_t)stream));
}

cfp32_status cfp32_cache_reserve(const int32_t *table, int64_t ld_table, const int32_t *lens, const int32_t *cu,
                                 const int32_t *refs, int32_t *table_out, int64_t ld_out, int32_t *refs_out,
                                 int32_t *missing, int64_t S, int64_t W, int64_t P, int64_t page, void *stream)
{
    const int lg = page_log2(page);
    if (!size_ok(S) || !size_ok(W) || !size_ok(P) || lg < 0 || W > (kMaxSize >> lg)) return CFP32_ERR_INVALID_VALUE;
    if (!table_ok(table, ld_table, S, W) || !table_ok(table_out, ld_out, S, W)) return CFP32_ERR_INVALID_VALUE;
    if ((S > 0 && (!lens || !cu)) || (P > 0 && (!refs || !refs_out))) return CFP32_ERR_INVALID_VALUE;
    if (table == table_out && ld_table != ld_out) return CFP32_ERR_INVALID_VALUE;
    if (S == 0 && P == 0 && !missing) return CFP32_OK;
    cfp32_status st = api_check_device();
    if (st != CFP32_OK) return st;
    return api_launched(cfp32::launch_cache_reserve(table, ld_table, lens, cu, refs, table_out, ld_out, refs_out, missing,
                                                    (int)S, (int)W, (int)P, lg, (hipStream_t)stream));
}

cfp32_status cfp32_cache_append(const float *k, int64_t k_tok, int64_t k_head, const float *v, int64_t v_tok,
                                int64_t v_head, const int32_t *cu, const int32_t *lens, int32_t *lens_out,
                                void *k_pages, int64_t kp_page, int64_t kp_head, int64_t kp_tok, void *v_pages,
                                int64_t vp_page, int64_t vp_head, int64_t vp_tok, int kv_type, int64_t P,
                                int64_t page, const int32_t *table, int64_t ld_table, int64_t S, int64_t W, int64_t T,
                                int64_t Hkv, int64_t D, void *stream)
{
    const int lg = page_log2(page);
    if (!size_ok(S) || !size_ok(W) || !size_ok(P) || !size_ok(T) || lg < 0 || W > (kMaxSize >> lg) ||
        !heads_ok(Hkv, Hkv, D) || !type_ok(kv_type))
        return CFP32_ERR_INVALID_VALUE;
    if (S == 0) return CFP32_OK;
    if (!cu || !lens || !lens_out || lens == lens_out || !table_ok(table, ld_table, S, W)) return CFP32_ERR_INVALID_VALUE;
    if (T > 0 && Hkv > 0 && D > 0) {
        if (!k || !v || !aligned_to(k, 4) || !aligned_to(v, 4)) return CFP32_ERR_INVALID_VALUE;
        if (!view_ok(T, k_tok, Hkv, k_head, 1, 0, D) || !view_ok(T, v_tok, Hkv, v_head, 1, 0, D))
            return CFP32_ERR_INVALID_VALUE;
        if (P > 0 && !pool_ok(k_pages, kp_page, kp_head, kp_tok, v_pages, vp_page, vp_head, vp_tok, P, Hkv, page, D,
                              kv_type, true))
            return CFP32_ERR_INVALID_VALUE;
    }
    cfp32_status st = api_check_device();
    if (st != CFP32_OK) return st;
    const cfp32::Pool pool = make_pool(k_pages, kp_page, kp_head, kp_tok, v_pages, vp_page, vp_head, vp_tok, P, page,
                                       Hkv, D, kv_type);
    return api_launched(cfp32::launch_cache_append({k, k_tok, k_head}, {v, v_tok, v_head}, cu, lens, lens_out, pool,
                                                   table, ld_table, (int)S, (int)W, (int)T, (hipStream_t)stream));
}

cfp32_status cfp32_cache_copy_pages(void *k_pages, int64_t kp_page, int64_t kp_head, int64_t kp_tok, void *v_pages,
                                    int64_t vp_page, int64_t vp_head, int64_t vp_tok, int kv_type, int64_t P,
                                    int64_t page, int64_t Hkv, int64_t D, const int32_t *src, const int32_t *dst,
                                    int64_t n, void *stream)
{
    if (!size_ok(P) || page_log2(page) < 0 || !heads_ok(Hkv, Hkv, D) || !type_ok(kv_type) || !size_ok(n))
        return CFP32_ERR_INVALID_VALUE;
    if (n == 0 || P == 0 || Hkv == 0 || D == 0) return CFP32_OK;
    if (!src || !dst || !pool_ok(k_pages, kp_page, kp_head, kp_tok, v_pages, vp_page, vp_head, vp_tok, P, Hkv, page, D,
                                 kv_type, true))
        return CFP32_ERR_INVALID_VALUE;
    cfp32_status st = api_check_device();
    if (st != CFP32_OK) return st;
    return api_launched(cfp32::launch_cache_copy_pages(make_pool(k_pages, kp_page, kp_head, kp_tok, v_pages, vp_page,
                                                                 vp_head, vp_tok, P, page, Hkv, D, kv_type),
                                                       src, dst, (int)n, (hipStream_t)stream));
}

size_t cfp32_cache_fork_workspace_bytes(int64_t C) { return size_ok(C) && C > 0 ? (size_t)C * 8 + kAlign : 0; }

cfp32_status cfp32_cache_fork(void *k_pages, int64_t kp_page, int64_t kp_head, int64_t kp_tok, void *v_pages,
                              int64_t vp_page, int64_t vp_head, int64_t vp_tok, int kv_type, int64_t P, int64_t page,
                              int64_t Hkv, int64_t D, const int32_t *table, int64_t ld_table, const int32_t *lens,
                              const int32_t *refs, const int32_t *parents, int32_t *table_out, int64_t ld_out,
                              int32_t *lens_out, int32_t *refs_out, int32_t *missing, int64_t S, int64_t W, int64_t C,
                              void *workspace, size_t workspace_bytes, void *stream)
{
    const int lg = page_log2(page);
    if (!size_ok(P) || lg < 0 || !heads_ok(Hkv, Hkv, D) || !type_ok(kv_type) || !size_ok(S) || !size_ok(W) ||
        !size_ok(C) || W > (kMaxSize >> lg))
        return CFP32_ERR_INVALID_VALUE;
    if ((P > 0 && (!refs || !refs_out)) || !table_ok(table, ld_table, S, W) || !table_ok(table_out, ld_out, C, W))
        return CFP32_ERR_INVALID_VALUE;
    if (P == 0 && C == 0 && !missing) return CFP32_OK;
    if (C > 0) {
        if (!parents || !lens_out || (S > 0 && !lens) || table_out == table || lens_out == lens)
            return CFP32_ERR_INVALID_VALUE;
        if (P > 0 && Hkv > 0 && D > 0 &&
            !pool_ok(k_pages, kp_page, kp_head, kp_tok, v_pages, vp_page, vp_head, vp_tok, P, Hkv, page, D, kv_type, true))
            return CFP32_ERR_INVALID_VALUE;
        if (!workspace || workspace_bytes < cfp32_cache_fork_workspace_bytes(C)) return CFP32_ERR_INVALID_VALUE;
    }
    cfp32_status st = api_check_device();
    if (st != CFP32_OK) return st;
    return api_launched(cfp32::launch_cache_fork(make_pool(k_pages, kp_page, kp_head, kp_tok, v_pages, vp_page, vp_head,
                                                           vp_tok, P, page, Hkv, D, kv_type),
                                                 table, ld_table, lens, refs, parents, table_out, ld_out, lens_out,
                                                 refs_out, missing, (int)S, (int)W, (int)C,
                                                 (int32_t *)align_up(workspace), (hipStream_t)stream));
}

cfp32_status cfp32_cache_free(const int32_t *rows, int64_t ld_rows, const int32_t *refs, int32_t *refs_out, int64_t R,
                              int64_t W, int64_t P, void *stream)
{
    if (!size_ok(R) || !size_ok(W) || !size_ok(P) || !table_ok(rows, ld_rows, R, W)) return CFP32_ERR_INVALID_VALUE;
    if (P == 0) return CFP32_OK;
    if (!refs || !refs_out) return CFP32_ERR_INVALID_VALUE;
    cfp32_status st = api_check_device();
    if (st != CFP32_OK) return st;
    return api_launched(cfp32::launch_cache_free(rows, ld_rows, refs, refs_out, (int)R, (int)W, (int)P, (hipStream_t)stream));
}

size_t cfp32_cache_compact_workspace_bytes(int64_t P) { return size_ok(P) && P > 0 ? (size_t)P * 12 + 4 + kAlign : 0; }

cfp32_status cfp32_cache_compact(void *k_pages, int64_t kp_page, int64_t kp_head, int64_t kp_tok, void *v_pages,
                                 int64_t vp_page, int64_t vp_head, int64_t vp_tok, int kv_type, int64_t P,
                                 int64_t page, int64_t Hkv, int64_t D, const int32_t *table, int64_t ld_table,
                                 const int32_t *refs, int32_t *table_out, int64_t ld_out, int32_t *refs_out,
                                 int32_t *live, int64_t S, int64_t W, void *workspace, size_t workspace_bytes,
                                 void *stream)
{
    if (!size_ok(P) || page_log2(page) < 0 || !heads_ok(Hkv, Hkv, D) || !type_ok(kv_type) || !size_ok(S) || !size_ok(W))
        return CFP32_ERR_INVALID_VALUE;
    if (!table_ok(table, ld_table, S, W) || !table_ok(table_out, ld_out, S, W) || !live) return CFP32_ERR_INVALID_VALUE;
    if (table == table_out && ld_table != ld_out) return CFP32_ERR_INVALID_VALUE;
    if (P > 0) {
        if (!refs || !refs_out || !workspace || workspace_bytes < cfp32_cache_compact_workspace_bytes(P))
            return CFP32_ERR_INVALID_VALUE;
        if (Hkv > 0 && D > 0 &&
            !pool_ok(k_pages, kp_page, kp_head, kp_tok, v_pages, vp_page, vp_head, vp_tok, P, Hkv, page, D, kv_type, true))
            return CFP32_ERR_INVALID_VALUE;
    }
    cfp32_status st = api_check_device();
    if (st != CFP32_OK) return st;
    return api_launched(cfp32::launch_cache_compact(make_pool(k_pages, kp_page, kp_head, kp_tok, v_pages, vp_page, vp_head,
                                                              vp_tok, P, page, Hkv, D, kv_type),
                                                    table, ld_table, refs, table_out, ld_out, refs_out, live, (int)S,
                                                    (int)W, (int32_t *)align_up(workspace), (hipStream_t)stream));
}

}  // extern "C"
