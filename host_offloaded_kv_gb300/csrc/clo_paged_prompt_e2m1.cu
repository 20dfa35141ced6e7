// Prompt attention over 4-bit pages.
#define CLO_PROMPT_BITS 4
#include "clo_paged_prompt.cu"
