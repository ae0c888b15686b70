// serve.hpp — launchers of the serving operators (mk_append_kv,
// mk_prompt_attention, mk_paged_attention, mk_process_logits).  Each takes
// arguments that check_* has accepted, enqueues on `stream` and returns MK_OK
// or MK_ERR_CUDA / MK_ERR_UNSUPPORTED with a message.
#pragma once
#include <string>

#include "../../include/mk.h"

namespace mk {
mk_status check_append(const mk_append_args& a, std::string& err);
mk_status check_prompt(const mk_prompt_args& a, std::string& err);
mk_status check_paged(const mk_paged_attn_args& a, std::string& err);
mk_status check_logits(const mk_logits_args& a, std::string& err);
size_t prompt_workspace_bytes(int batch, int n_tokens, int n_q_heads, int n_kv_heads, int head_dim, long long max_keys);
size_t paged_workspace_bytes(int batch, int n_q_heads, int n_kv_heads, int head_dim);

mk_status launch_append(const mk_append_args& a, void* stream, std::string& err);
mk_status launch_prompt(const mk_prompt_args& a, void* stream, std::string& err);
mk_status launch_paged(const mk_paged_attn_args& a, void* stream, std::string& err);
mk_status launch_logits(const mk_logits_args& a, void* stream, std::string& err);
}  // namespace mk
