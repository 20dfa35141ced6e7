// Prompt attention over 8-bit pages.
#define CLO_PROMPT_BITS 8
#include "clo_paged_prompt.cu"
