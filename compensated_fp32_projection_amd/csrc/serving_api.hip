// C ABI of the rotary, 8-bit cache and beam calls (declared in
// include/cfp32.h): argument validation, the device check and workspace sizes.
// Every call validates all of its arguments before it enqueues anything.
#include "api_checks.h"
#include "attention8.h"
#include "beam.h"
#include "rotary.h"

namespace {

using namespace cfp32;

// In place, or apart (which the caller sees to).
bool same_view(const void *in, int64_t s0, int64_t s1, const void *out, int64_t o0, int64_t o1)
{
    return in != out || (s0 == o0 && s1 == o1);
}

// An 8-bit cache: sizes, and (written: or) pools that are only read.
bool sizes_ok(const cfp32_cache8 *c)
{
    if (!c || !size_ok(c->P) || page_log2(c->page) < 0 || page_log2(c->block) < 0 || c->block > c->page) return false;
    if (!heads_ok(c->Hkv, c->Hkv, c->D) || c->Hkv > 65535) return false;  // a token's values are counted in 32 bits
    return c->code_type == CFP32_CODE_I8 || c->code_type == CFP32_CODE_E4M3;
}

bool pools_ok(const cfp32_cache8 *c, bool written)
{
    if (c->P == 0 || c->Hkv == 0 || c->D == 0) return true;
    const int64_t P = c->P, H = c->Hkv, blocks = c->page / c->block;
    if (!c->k || !c->v || !c->k_scales || !c->v_scales || !aligned_to(c->k_scales, 4) || !aligned_to(c->v_scales, 4)) return false;
    auto ok = [&](int64_t s1, int64_t s2, int64_t n3, int64_t s3, int64_t n) {
        return view_ok(P, s1, H, s2, n3, s3, n) && (!written || distinct_ok(P, s1, H, s2, n3, s3, n));
    };
    return ok(c->k_page, c->k_head, c->page, c->k_tok, c->D) && ok(c->v_page, c->v_head, c->page, c->v_tok, c->D) &&
           ok(c->ks_page, c->ks_head, 1, 0, blocks) && ok(c->vs_page, c->vs_head, 1, 0, blocks);
}

Cache8 view_of(const cfp32_cache8 *c)
{
    return {{c->k, c->k_page, c->k_head, c->k_tok}, {c->v, c->v_page, c->v_head, c->v_tok}, {c->k_scales, c->ks_page, c->ks_head},
            {c->v_scales, c->vs_page, c->vs_head}, (int)c->P, (int)c->Hkv, (int)c->D, page_log2(c->page), page_log2(c->block),
            c->code_type == CFP32_CODE_E4M3};
}

// Its codes and its scales (a page's are one value wide) as pools of pages to be moved.
Pool codes_of(const cfp32_cache8 *c)
{
    return {{c->k, c->k_page, c->k_head, c->k_tok}, {c->v, c->v_page, c->v_head, c->v_tok}, (int)c->P, page_log2(c->page),
            (int)c->Hkv, (int)c->D, 1};
}
Pool scales_of(const cfp32_cache8 *c)
{
    return {{c->k_scales, c->ks_page, c->ks_head, 1}, {c->v_scales, c->vs_page, c->vs_head, 1}, (int)c->P,
            page_log2(c->page) - page_log2(c->block), (int)c->Hkv, c->D > 0 ? 1 : 0, 4};
}

}  // namespace

extern "C" {

cfp32_status cfp32_rotary_frequencies(double theta, int64_t R, int scaling, double factor, double trained, double slow,
                                      double fast, double *frequencies, double *amplitude)
{
    if (!(theta > 0.0) || !std::isfinite(theta) || R < 2 || R % 2 || R > kRotaryMaxDim || !frequencies || !amplitude)
        return CFP32_ERR_INVALID_VALUE;
    if (scaling < CFP32_ROTARY_PLAIN || scaling > CFP32_ROTARY_PARTS) return CFP32_ERR_INVALID_VALUE;
    if (scaling != CFP32_ROTARY_PLAIN && !(factor >= 1.0 && std::isfinite(factor))) return CFP32_ERR_INVALID_VALUE;
    if (scaling == CFP32_ROTARY_PARTS &&
        !(trained > 0.0 && std::isfinite(trained) && std::isfinite(slow) && std::isfinite(fast) && slow < fast))
        return CFP32_ERR_INVALID_VALUE;
    const double n = (double)R;
    if (scaling == CFP32_ROTARY_NTK && R > 2) theta *= std::pow(factor, n / (n - 2.0));
    if (!std::isfinite(theta)) return CFP32_ERR_INVALID_VALUE;
    for (int64_t i = 0; i < R / 2; ++i) {
        double f = std::pow(theta, -2.0 * (double)i / n);
        if (scaling == CFP32_ROTARY_LINEAR) f /= factor;
        if (scaling == CFP32_ROTARY_PARTS) {
            const double turns = trained * f / 6.283185307179586476925286766559;
            const double g = std::fmin(std::fmax((turns - slow) / (fast - slow), 0.0), 1.0);
            f = g * f + (1.0 - g) * f / factor;
        }
        frequencies[i] = f;
    }
    *amplitude = scaling == CFP32_ROTARY_PARTS ? 1.0 + 0.1 * std::log(factor) : 1.0;
    return CFP32_OK;
}

cfp32_status cfp32_rotary(const void *q, int64_t q_tok, int64_t q_head, const void *k, int64_t k_tok, int64_t k_head, int type,
                          const int64_t *positions, const double *frequencies, double amplitude, int layout, int transpose,
                          void *q_out, int64_t qo_tok, int64_t qo_head, void *k_out, int64_t ko_tok, int64_t ko_head,
                          int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t R, void *stream)
{
    if (!size_ok(T) || !size_ok(Hq) || !size_ok(Hkv) || D < 0 || D > kRotaryMaxDim || R < 0 || R > D || R % 2 || !type_ok(type))
        return CFP32_ERR_INVALID_VALUE;
    if (Hq + Hkv > kMaxSize / kRotaryMaxDim) return CFP32_ERR_INVALID_VALUE;  // a token's items are counted in 32 bits
    if (layout != CFP32_ROTARY_HALF && layout != CFP32_ROTARY_INTERLEAVED) return CFP32_ERR_INVALID_VALUE;
    if (!scale_ok(amplitude)) return CFP32_ERR_INVALID_VALUE;
    if (T == 0 || D == 0 || Hq + Hkv == 0) return CFP32_OK;
    const size_t al = type == CFP32_KV_F16 ? 2 : 4;
    auto ok = [&](const void *in, int64_t s0, int64_t s1, const void *out, int64_t o0, int64_t o1, int64_t H) {
        return H == 0 || (in && out && aligned_to(in, al) && aligned_to(out, al) && view_ok(T, s0, H, s1, 1, 0, D) &&
                          view_ok(T, o0, H, o1, 1, 0, D) && distinct_ok(T, o0, H, o1, 1, 0, D) &&
                          same_view(in, s0, s1, out, o0, o1));
    };
    if (!ok(q, q_tok, q_head, q_out, qo_tok, qo_head, Hq) || !ok(k, k_tok, k_head, k_out, ko_tok, ko_head, Hkv))
        return CFP32_ERR_INVALID_VALUE;
    // Rows that another thread reads or writes, too.
    if (Hq > 0 && Hkv > 0 && q != k && (q_out == k_out || q_out == k || k_out == q)) return CFP32_ERR_INVALID_VALUE;
    if ((R > 0 && !frequencies) || !aligned_to(frequencies, 8) || !aligned_to(positions, 8)) return CFP32_ERR_INVALID_VALUE;
    cfp32_status st = api_check_device();
    if (st != CFP32_OK) return st;
    const RotaryArgs a = {{q, q_out, q_tok, q_head, qo_tok, qo_head, (int)Hq}, {k, k_out, k_tok, k_head, ko_tok, ko_head, (int)Hkv},
                          positions, frequencies, (float)amplitude, type == CFP32_KV_F16, layout == CFP32_ROTARY_INTERLEAVED,
                          transpose != 0, (int)T, (int)D, (int)R};
    return api_launched(launch_rotary(a, (hipStream_t)stream));
}

cfp32_status cfp32_cache8_append(const float *k, int64_t k_tok, int64_t k_head, const float *v, int64_t v_tok, int64_t v_head,
                                 const int32_t *cu, const int32_t *lens, int32_t *lens_out, const cfp32_cache8 *cache,
                                 const int32_t *table, int64_t ld_table, int64_t S, int64_t W, int64_t T, void *stream)
{
    if (!sizes_ok(cache) || !size_ok(S) || !size_ok(W) || !size_ok(T) || W > (kMaxSize >> page_log2(cache->page)))
        return CFP32_ERR_INVALID_VALUE;
    if (S == 0) return CFP32_OK;
    if (!cu || !lens || !lens_out || lens == lens_out || !table_ok(table, ld_table, S, W)) return CFP32_ERR_INVALID_VALUE;
    const int64_t H = cache->Hkv, D = cache->D;
    if (T > 0 && H > 0 && D > 0) {
        if (!k || !v || !aligned_to(k, 4) || !aligned_to(v, 4) || !view_ok(T, k_tok, H, k_head, 1, 0, D) ||
            !view_ok(T, v_tok, H, v_head, 1, 0, D) || !pools_ok(cache, true))
            return CFP32_ERR_INVALID_VALUE;
    }
    cfp32_status st = api_check_device();
    if (st != CFP32_OK) return st;
    return api_launched(launch_cache8_append({k, k_tok, k_head}, {v, v_tok, v_head}, cu, lens, lens_out, view_of(cache), table,
                                             ld_table, (int)S, (int)W, (int)T, (hipStream_t)stream));
}

cfp32_status cfp32_cache8_read(const cfp32_cache8 *cache, const int32_t *table, int64_t ld_table, const int32_t *first,
                               const int32_t *cu, void *k, int64_t k_tok, int64_t k_head, void *v, int64_t v_tok, int64_t v_head,
                               int out_type, int64_t S, int64_t W, int64_t T, void *stream)
{
    if (!sizes_ok(cache) || !type_ok(out_type) || !size_ok(S) || !size_ok(W) || !size_ok(T) ||
        W > (kMaxSize >> page_log2(cache->page)))
        return CFP32_ERR_INVALID_VALUE;
    const int64_t H = cache->Hkv, D = cache->D;
    if (S == 0 || T == 0 || H == 0 || D == 0) return CFP32_OK;
    const size_t al = out_type == CFP32_KV_F16 ? 2 : 4;
    if (!cu || !k || !v || !aligned_to(k, al) || !aligned_to(v, al) || !table_ok(table, ld_table, S, W, true) || !pools_ok(cache, false))
        return CFP32_ERR_INVALID_VALUE;
    if (!view_ok(T, k_tok, H, k_head, 1, 0, D) || !view_ok(T, v_tok, H, v_head, 1, 0, D) ||
        !distinct_ok(T, k_tok, H, k_head, 1, 0, D) || !distinct_ok(T, v_tok, H, v_head, 1, 0, D))
        return CFP32_ERR_INVALID_VALUE;
    cfp32_status st = api_check_device();
    if (st != CFP32_OK) return st;
    return api_launched(launch_cache8_read(view_of(cache), table, ld_table, first, cu, {k, k_tok, k_head}, {v, v_tok, v_head},
                                           out_type == CFP32_KV_F16, (int)S, (int)W, (int)T, (hipStream_t)stream));
}

cfp32_status cfp32_cache8_copy_pages(const cfp32_cache8 *cache, const int32_t *src, const int32_t *dst, int64_t n, void *stream)
{
    if (!sizes_ok(cache) || !size_ok(n)) return CFP32_ERR_INVALID_VALUE;
    if (n == 0 || cache->P == 0 || cache->Hkv == 0 || cache->D == 0) return CFP32_OK;
    if (!src || !dst || !pools_ok(cache, true)) return CFP32_ERR_INVALID_VALUE;
    cfp32_status st = api_check_device();
    if (st != CFP32_OK) return st;
    return api_launched(launch_cache8_copy_pages(codes_of(cache), scales_of(cache), src, dst, (int)n, (hipStream_t)stream));
}

cfp32_status cfp32_cache8_fork(const cfp32_cache8 *cache, const int32_t *table, int64_t ld_table, const int32_t *lens,
                               const int32_t *refs, const int32_t *parents, int32_t *table_out, int64_t ld_out, int32_t *lens_out,
                               int32_t *refs_out, int32_t *missing, int64_t S, int64_t W, int64_t C, void *workspace,
                               size_t workspace_bytes, void *stream)
{
    if (!sizes_ok(cache) || !size_ok(S) || !size_ok(W) || !size_ok(C) || W > (kMaxSize >> page_log2(cache->page)))
        return CFP32_ERR_INVALID_VALUE;
    if ((cache->P > 0 && (!refs || !refs_out)) || !table_ok(table, ld_table, S, W) || !table_ok(table_out, ld_out, C, W))
        return CFP32_ERR_INVALID_VALUE;
    if (cache->P == 0 && C == 0 && !missing) return CFP32_OK;
    if (C > 0) {
        if (!parents || !lens_out || (S > 0 && !lens) || table_out == table || lens_out == lens || !pools_ok(cache, true))
            return CFP32_ERR_INVALID_VALUE;
        if (!workspace || workspace_bytes < cfp32_cache_fork_workspace_bytes(C)) return CFP32_ERR_INVALID_VALUE;
    }
    cfp32_status st = api_check_device();
    if (st != CFP32_OK) return st;
    return api_launched(launch_cache8_fork(codes_of(cache), scales_of(cache), table, ld_table, lens, refs, parents, table_out,
                                           ld_out, lens_out, refs_out, missing, (int)S, (int)W, (int)C,
                                           (int32_t *)align_up(workspace), (hipStream_t)stream));
}

cfp32_status cfp32_cache8_compact(const cfp32_cache8 *cache, const int32_t *table, int64_t ld_table, const int32_t *refs,
                                  int32_t *table_out, int64_t ld_out, int32_t *refs_out, int32_t *live, int64_t S, int64_t W,
                                  void *workspace, size_t workspace_bytes, void *stream)
{
    if (!sizes_ok(cache) || !size_ok(S) || !size_ok(W)) return CFP32_ERR_INVALID_VALUE;
    if (!table_ok(table, ld_table, S, W) || !table_ok(table_out, ld_out, S, W) || !live) return CFP32_ERR_INVALID_VALUE;
    if (table == table_out && ld_table != ld_out) return CFP32_ERR_INVALID_VALUE;
    if (cache->P > 0 && (!refs || !refs_out || !workspace ||
                         workspace_bytes < cfp32_cache_compact_workspace_bytes(cache->P) || !pools_ok(cache, true)))
        return CFP32_ERR_INVALID_VALUE;
    cfp32_status st = api_check_device();
    if (st != CFP32_OK) return st;
    return api_launched(launch_cache8_compact(codes_of(cache), scales_of(cache), table, ld_table, refs, table_out, ld_out, refs_out,
                                              live, (int)S, (int)W, (int32_t *)align_up(workspace), (hipStream_t)stream));
}

size_t cfp32_attention8_decode_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t W, int64_t page)
{
    const int lg = page_log2(page);
    if (!size_ok(B) || !heads_ok(Hq, Hkv, D) || Hkv > 65535 || !size_ok(W) || lg < 0 || W > (kMaxKeys >> lg)) return 0;
    if (B == 0 || Hq == 0 || D == 0 || B > (kMaxDim >> 20) / Hq) return 0;
    const size_t n = attention8_decode_workspace(B, Hq, Hkv, D, W, lg);
    return n ? n + kAlign : 0;
}

cfp32_status cfp32_attention8_decode(const float *q, int64_t q_seq, int64_t q_head, const cfp32_cache8 *cache,
                                     const int32_t *table, int64_t ld_table, int64_t W, const int32_t *lens, float *out,
                                     int64_t out_seq, int64_t out_head, int64_t B, int64_t Hq, double scale, void *workspace,
                                     size_t workspace_bytes, void *stream)
{
    if (!sizes_ok(cache) || !size_ok(B) || !heads_ok(Hq, cache->Hkv, cache->D) || !size_ok(W) ||
        W > (kMaxKeys >> page_log2(cache->page)))
        return CFP32_ERR_INVALID_VALUE;
    const int64_t D = cache->D;
    if (B == 0 || Hq == 0 || D == 0) return CFP32_OK;
    if (B > (kMaxDim >> 20) / Hq) return CFP32_ERR_INVALID_VALUE;
    if (!q || !out || !lens || !table_ok(table, ld_table, B, W, true) || !pools_ok(cache, false)) return CFP32_ERR_INVALID_VALUE;
    if (!aligned_to(q, 4) || !aligned_to(out, 4) || !view_ok(B, q_seq, Hq, q_head, 1, 0, D) ||
        !view_ok(B, out_seq, Hq, out_head, 1, 0, D) || !distinct_ok(B, out_seq, Hq, out_head, 1, 0, D))
        return CFP32_ERR_INVALID_VALUE;
    if (!scale_ok(scale)) return CFP32_ERR_INVALID_VALUE;
    const size_t need = cfp32_attention8_decode_workspace_bytes(B, Hq, cache->Hkv, D, W, cache->page);
    if (need && (!workspace || workspace_bytes < need)) return CFP32_ERR_INVALID_VALUE;
    cfp32_status st = api_check_device();
    if (st != CFP32_OK) return st;
    const Decode8Args a = {q, q_seq, q_head, view_of(cache), table, ld_table, lens, out, out_seq, out_head, (int)B, (int)Hq,
                           (int)W, (float)scale};
    return api_launched(launch_attention8_decode(a, align_up(workspace), (hipStream_t)stream));
}

size_t cfp32_beam_select_workspace_bytes(int64_t S, int64_t beams, int64_t V, int64_t n)
{
    if (!size_ok(S) || beams < 1 || beams > kMaxBeams || n < 1 || n > kMaxBeams || V < 1 || V > kMaxSize - 4096) return 0;
    if (S == 0 || S > kMaxSize / kMaxBeams) return 0;
    return plan_beam(S, beams, V, n).bytes + kAlign;
}

cfp32_status cfp32_beam_select(const float *logits, int64_t ld, const float *scores, const uint8_t *done, int64_t S,
                               int64_t beams, int64_t V, int64_t n, int64_t eos, int32_t *parents, int32_t *tokens,
                               float *scores_out, uint8_t *done_out, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!size_ok(S) || S > kMaxSize / kMaxBeams || beams < 1 || beams > kMaxBeams || n < 1 || n > kMaxBeams || V < 1 ||
        V > kMaxSize - 4096 || (ld < V && ld) || eos < -kMaxSize || eos > kMaxSize)
        return CFP32_ERR_INVALID_VALUE;
    if (S == 0) return CFP32_OK;
    if (!logits || !scores || !parents || !tokens || !scores_out || !aligned_to(logits, 4) || !view_ok(S * beams, ld, 1, 0, 1, 0, V))
        return CFP32_ERR_INVALID_VALUE;
    if (scores_out == scores || (done && done_out == done)) return CFP32_ERR_INVALID_VALUE;  // a block reads what others write
    if (!workspace || workspace_bytes < cfp32_beam_select_workspace_bytes(S, beams, V, n)) return CFP32_ERR_INVALID_VALUE;
    cfp32_status st = api_check_device();
    if (st != CFP32_OK) return st;
    const BeamArgs a = {logits, ld, scores, done, (int)S, (int)beams, (int)V, (int)n, (int)eos, parents, tokens, scores_out, done_out};
    return api_launched(launch_beam_select(a, align_up(workspace), (hipStream_t)stream));
}

cfp32_status cfp32_beam_reorder(const void *states, int64_t stride, void *out, int64_t out_stride, const int32_t *parents,
                                int64_t rows, int64_t n, int64_t row_bytes, void *stream)
{
    if (!size_ok(rows) || !size_ok(n) || row_bytes < 0 || row_bytes > kMaxDim || !term_ok(rows, stride) || out_stride < row_bytes ||
        !term_ok(n, out_stride) || (n > 0 && row_bytes > kMaxDim / n))
        return CFP32_ERR_INVALID_VALUE;
    if (n == 0 || row_bytes == 0) return CFP32_OK;
    if ((rows > 0 && !states) || !out || !parents || out == states) return CFP32_ERR_INVALID_VALUE;
    cfp32_status st = api_check_device();
    if (st != CFP32_OK) return st;
    return api_launched(launch_beam_reorder(states, stride, out, out_stride, parents, (int)rows, (int)n, row_bytes,
                                            (hipStream_t)stream));
}

}  // extern "C"
